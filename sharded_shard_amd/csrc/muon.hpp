// Kernel launchers of the Muon momentum and update on fp32 shards.  Each
// enqueues one kernel over a plan's copy-in tiles on `st` and returns
// hipGetLastError(); n is the number of tiles, and n == 0 launches nothing.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "plan.hpp"

namespace fsdp {

// momentum from the grad shards, its update into the bf16 segment ag_in;
// scal: mu, 1 - mu
hipError_t launch_muon_momentum(const PackTile *tiles, int64_t n, const DevEntry *ents,
                                uint16_t *ag_in, const float scal[2], bool nesterov,
                                hipStream_t st);
// the same from the mean of the N rows of rs_in ([N, S] bf16); chunk_aligned:
// every row piece starts 16-byte aligned
hipError_t launch_muon_reduce_momentum(const PackTile *tiles, int64_t n, const DevEntry *ents,
                                       const uint16_t *rs_in, uint16_t *ag_in, int64_t S,
                                       int32_t N, const float scal[2], bool nesterov,
                                       bool chunk_aligned, hipStream_t st);
// update of the master shards by upd (a bf16 segment, or with null the rank's
// rows of the bound full tensors, which start own[entry] elements into them);
// scales: one fp32 per parameter, or null for 1; ag_in: the copy-in segment,
// or null; scal: 1 - lr*wd, lr
hipError_t launch_muon_update(const PackTile *tiles, int64_t n, const DevEntry *ents,
                              const int64_t *own, const uint16_t *upd, uint16_t *ag_in,
                              const float *scales, const float scal[2], hipStream_t st);

}  // namespace fsdp
