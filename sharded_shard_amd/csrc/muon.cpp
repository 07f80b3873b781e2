// C ABI of the Muon momentum and update: argument checks, then one launch.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "../../include/fsdp_shard.h"
#include "muon.hpp"
#include "state.hpp"

namespace {

using fsdp::set_error;

// [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) &&
           y < x + static_cast<uintptr_t>(na);
}

int64_t segment_bytes(const fsdp_plan *p) { return p->L.S * 2; }

// No byte of buf is part of a bound shard that the call reads or writes.
fsdp_status check_apart(const fsdp_plan *p, const void *buf, int64_t bytes, int32_t roles,
                        const char *call, const char *name) {
    for (size_t i = 0; i < p->L.entries.size(); ++i) {
        const fsdp_shard_entry_t &t = p->L.entries[i];
        const fsdp::DevEntry &e = p->host_entries[i];
        if (((roles & FSDP_ROLE_MASTER) && overlap(buf, bytes, e.master, t.valid_numel * 4)) ||
            ((roles & FSDP_ROLE_GRAD) && overlap(buf, bytes, e.grad, t.valid_numel * 4)) ||
            ((roles & FSDP_ROLE_EXP_AVG) && overlap(buf, bytes, e.exp_avg, t.valid_numel * 4)) ||
            ((roles & FSDP_ROLE_FULL) && overlap(buf, bytes, e.full, t.rows * t.cols * 2)))
            return set_error(FSDP_E_INVAL, std::string(call) + ": " + name +
                                               " overlaps a bound tensor of parameter " +
                                               std::to_string(i));
    }
    return FSDP_OK;
}

fsdp_status check_momentum(const fsdp_muon_hparams_t *hp, const char *call) {
    if (hp == nullptr) return set_error(FSDP_E_INVAL, std::string(call) + ": null hyperparameters");
    if (!(hp->momentum >= 0.0 && hp->momentum < 1.0))
        return set_error(FSDP_E_INVAL, std::string(call) + ": momentum must lie in [0, 1)");
    return FSDP_OK;
}

// mu and 1 - mu, from fp64, rounded once.
void momentum_scalars(const fsdp_muon_hparams_t *hp, float out[2]) {
    out[0] = static_cast<float>(hp->momentum);
    out[1] = static_cast<float>(1.0 - hp->momentum);
}

fsdp_status launched(hipError_t e, const char *call) {
    return e == hipSuccess ? FSDP_OK
                           : fsdp::set_hip_error(e, (std::string(call) + ": launch").c_str());
}

}  // namespace

extern "C" {

fsdp_status fsdp_muon_momentum(const fsdp_plan *p, uint16_t *ag_in, const fsdp_muon_hparams_t *hp,
                               void *stream) try {
    const char *call = "fsdp_muon_momentum";
    const int32_t roles = FSDP_ROLE_GRAD | FSDP_ROLE_EXP_AVG;
    fsdp_status s = fsdp::check_roles(p, roles, call);
    if (s != FSDP_OK || (s = fsdp::check_segment(p, ag_in, call, "ag_in")) != FSDP_OK ||
        (s = check_momentum(hp, call)) != FSDP_OK ||
        (s = check_apart(p, ag_in, segment_bytes(p), roles, call, "ag_in")) != FSDP_OK ||
        (s = fsdp::check_plan_device(p)) != FSDP_OK)
        return s;
    float scal[2];
    momentum_scalars(hp, scal);
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_muon_momentum(p->d_pack, static_cast<int64_t>(p->L.pack.size()),
                                       p->d_entries, ag_in, scal, hp->nesterov != 0,
                                       static_cast<hipStream_t>(stream));
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_muon_reduce_momentum(const fsdp_plan *p, const uint16_t *rs_in, uint16_t *ag_in,
                                      const fsdp_muon_hparams_t *hp, void *stream) try {
    const char *call = "fsdp_muon_reduce_momentum";
    fsdp_status s = fsdp::check_roles(p, FSDP_ROLE_EXP_AVG, call);
    if (s != FSDP_OK || (s = fsdp::check_segment(p, rs_in, call, "rs_in")) != FSDP_OK ||
        (s = fsdp::check_segment(p, ag_in, call, "ag_in")) != FSDP_OK ||
        (s = check_momentum(hp, call)) != FSDP_OK)
        return s;
    const int64_t rows = segment_bytes(p) * p->L.world;
    if (overlap(ag_in, segment_bytes(p), rs_in, rows))
        return set_error(FSDP_E_INVAL, std::string(call) + ": ag_in overlaps rs_in");
    if ((s = check_apart(p, ag_in, segment_bytes(p), FSDP_ROLE_EXP_AVG, call, "ag_in")) !=
            FSDP_OK ||
        (s = check_apart(p, rs_in, rows, FSDP_ROLE_EXP_AVG, call, "rs_in")) != FSDP_OK ||
        (s = fsdp::check_plan_device(p)) != FSDP_OK)
        return s;
    float scal[2];
    momentum_scalars(hp, scal);
    const bool aligned = p->L.offsets8 && (reinterpret_cast<uintptr_t>(rs_in) & 15u) == 0;
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_muon_reduce_momentum(
            p->d_pack, static_cast<int64_t>(p->L.pack.size()), p->d_entries, rs_in, ag_in, p->L.S,
            p->L.world, scal, hp->nesterov != 0, aligned, static_cast<hipStream_t>(stream));
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_muon_update(const fsdp_plan *p, const uint16_t *upd, uint16_t *ag_in,
                             const float *scales, const fsdp_muon_hparams_t *hp,
                             void *stream) try {
    const char *call = "fsdp_muon_update";
    // without a segment the update is read from the rank's rows of the full tensors
    // (an empty segment has no address)
    const bool rows = upd == nullptr && p != nullptr && p->L.S > 0;
    const int32_t roles = FSDP_ROLE_MASTER | (rows ? FSDP_ROLE_FULL : 0);
    fsdp_status s = fsdp::check_roles(p, roles, call);
    if (s != FSDP_OK) return s;
    if (hp == nullptr) return set_error(FSDP_E_INVAL, std::string(call) + ": null hyperparameters");
    if (!std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay))
        return set_error(FSDP_E_INVAL, std::string(call) + ": lr or weight_decay is not finite");
    if ((reinterpret_cast<uintptr_t>(scales) & 3u) != 0)
        return set_error(FSDP_E_ALIGN, std::string(call) + ": scales not 4-byte aligned");
    const int64_t n_scales = static_cast<int64_t>(p->L.entries.size()) * 4;
    if (scales != nullptr &&
        (s = check_apart(p, scales, n_scales, FSDP_ROLE_MASTER, call, "scales")) != FSDP_OK)
        return s;
    if (upd != nullptr) {
        if ((s = fsdp::check_segment(p, upd, call, "upd")) != FSDP_OK ||
            (s = check_apart(p, upd, segment_bytes(p), roles, call, "upd")) != FSDP_OK)
            return s;
    }
    if (ag_in != nullptr) {
        if ((s = fsdp::check_segment(p, ag_in, call, "ag_in")) != FSDP_OK ||
            (s = check_apart(p, ag_in, segment_bytes(p), roles, call, "ag_in")) != FSDP_OK)
            return s;
        if (overlap(ag_in, segment_bytes(p), upd, upd != nullptr ? segment_bytes(p) : 0))
            return set_error(FSDP_E_INVAL, std::string(call) + ": ag_in overlaps upd");
        if (scales != nullptr && overlap(ag_in, segment_bytes(p), scales, n_scales))
            return set_error(FSDP_E_INVAL, std::string(call) + ": ag_in overlaps scales");
    }
    if ((s = fsdp::check_plan_device(p)) != FSDP_OK) return s;
    const float scal[2] = {static_cast<float>(1.0 - hp->lr * hp->weight_decay),
                           static_cast<float>(hp->lr)};
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_muon_update(p->d_pack, static_cast<int64_t>(p->L.pack.size()),
                                     p->d_entries, p->d_own, upd, ag_in, scales, scal,
                                     static_cast<hipStream_t>(stream));
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

}  // extern "C"
