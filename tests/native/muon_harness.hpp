// Shared between the Muon sanitizer harness and its launch stand-ins.
#pragma once

#include <cstdint>
#include <vector>

#include "../../sharded_shard_amd/csrc/ortho.hpp"

namespace harness {

enum { kNorm = 0, kInit, kGram, kJoin, kPoly, kApply, kLast, kSums, kSmall /* + mode */ };

struct Launch {
    int what;
    int32_t tile, split;
    std::vector<fsdp::OrthoTile> tiles;
};

struct Written {
    const void *base;
    int64_t off, len;
};

extern std::vector<Launch> ortho;   // since the last clear
extern std::vector<Written> muon;

}  // namespace harness
