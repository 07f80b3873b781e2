// The plan behind the C ABI's opaque handle, and the argument checks and error
// reporting that its translation units share (defined in capi.cpp).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <string>
#include <vector>

#include "../../include/fsdp_shard.h"
#include "plan.hpp"
#include "q8.hpp"

struct fsdp_plan {
    fsdp::Layout L;
    std::vector<fsdp::DevEntry> host_entries;
    int32_t bound = 0;
    int device = -1;
    bool tiles_uploaded = false;  // the tile tables below hold the plan's tiles
    char *dmem = nullptr;  // one device block: entries, then the tile tables
    fsdp::DevEntry *d_entries = nullptr;
    fsdp::PackTile *d_pack = nullptr;
    fsdp::PackTile *d_rspack = nullptr;
    fsdp::UnpackTile *d_unpack = nullptr;
    fsdp::ReduceTile *d_reduce = nullptr;
    fsdp::EwTile *d_adamw = nullptr;
    fsdp::EwTile *d_full = nullptr;
    int64_t *d_own = nullptr;     // per parameter: element offset of this rank's rows
    fsdp::BlockEntry *d_blocks = nullptr;   // per parameter: its 128 x 128 blocks
    fsdp::BlockCell *d_cells = nullptr;     // this rank's part of each block
    int64_t n_cells = 0, n_block_scales = 0;
};

namespace fsdp {

// Records a failed call's message for fsdp_last_error and returns its status.
fsdp_status set_error(fsdp_status s, const std::string &msg);
fsdp_status set_hip_error(hipError_t e, const char *what);
// hipSuccess, or the failure that FSDP_FAULT asks for in place of a launch.
hipError_t injected_fault();
// The plan exists and holds the tensors of `roles`.
fsdp_status check_roles(const fsdp_plan *p, int32_t roles, const char *call);
// The current device is the one the plan's tables live on.
fsdp_status check_plan_device(const fsdp_plan *p);
// A bf16 segment buffer: present where the plan has elements, 2-byte aligned.
fsdp_status check_segment(const fsdp_plan *p, const void *buf, const char *call, const char *name);

}  // namespace fsdp
