"""Host-side checks of the Muon momentum and update: the oracle's pins and the
library's refusals (no GPU needed)."""
import numpy as np
import pytest

from oracle import fsdp as O
from oracle import muon as M

capi = pytest.importorskip("sharded_shard_amd.capi")

SHAPES = [(5, 3), (0, 4), (1, 5), (13, 2)]


def _shards(p, seed):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(e.valid_numel).astype(np.float32) for e in p.entries]


# ---- the oracle against formulas that it does not use ---------------------------

@pytest.mark.parametrize("nesterov", [False, True])
def test_momentum_is_the_exponential_average_of_the_gradients(nesterov):
    """From m = 0, m_t = (1-mu) sum_k mu^(t-k) g_k, and u = m or the same
    average taken one step further with g_t in the place of the next gradient.
    Each of t steps rounds three times (half a step of 2^-24 each, relative to
    partial sums that |g| bounds), the bf16 output once more (2^-8 / 2)."""
    p = O.plan(SHAPES, 2, 0)
    mu, steps = 0.9, 4
    ms = [np.zeros(e.valid_numel, np.float32) for e in p.entries]
    gs = [_shards(p, k) for k in range(steps)]
    for g in gs:
        seg = M.momentum(p, g, ms, mu, nesterov)
    for i, e in enumerate(p.entries):
        n, o = e.valid_numel, e.shard_offset
        want = sum((1 - mu) * mu ** (steps - 1 - k) * gs[k][i].astype(np.float64)
                   for k in range(steps))
        big = sum(np.abs(gs[k][i]).astype(np.float64) for k in range(steps))
        assert (np.abs(ms[i] - want) <= 4 * steps * 2.0 ** -24 * big).all()
        u = mu * want + (1 - mu) * gs[-1][i] if nesterov else want
        err = np.abs(O.bf16_to_f32(seg[o:o + n]) - u)
        assert (err <= 2.0 ** -8 * np.abs(u) + 8 * steps * 2.0 ** -24 * big).all()
        assert (seg[o + n:o + e.seg_numel] == 0).all()


def test_update_is_decay_then_step():
    p = O.plan(SHAPES, 2, 1)
    xs = _shards(p, 7)
    was = [x.astype(np.float64) for x in xs]
    upd = [O.bf16_rne(o) for o in _shards(p, 8)]
    scales, lr, wd = [1.5, 1.0, 0.25, 2.0], 0.02, 0.1
    seg = M.update(p, xs, upd, scales, lr, wd)
    for x, x0, o, s, e in zip(xs, was, upd, scales, p.entries):
        want = x0 - lr * wd * x0 - lr * s * O.bf16_to_f32(o)
        assert (np.abs(x - want) <= 2.0 ** -22 * (np.abs(x0) + np.abs(want) + 0.1)).all()
        assert np.array_equal(seg[e.shard_offset:e.shard_offset + e.valid_numel], O.bf16_rne(x))


@pytest.mark.parametrize("shape", [(1, 7), (7, 1), (4, 9), (9, 4), (6, 6)])
def test_orthogonalize_maps_the_singular_values(shape):
    """X_k = U f_k(...f_1(S)) V^T with f(s) = a s + b s^3 + c s^5."""
    coeffs = [(3.4445, -4.7750, 2.0315)] * 5
    u = np.random.default_rng(shape[0]).standard_normal(shape)
    got = M.orthogonalize(u, coeffs)
    left, s, right = np.linalg.svd(u, full_matrices=False)
    s = s / (np.sqrt((u * u).sum()) + 1e-7)
    for a, b, c in coeffs:
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(got, left @ np.diag(s) @ right, atol=1e-11)
    assert (M.orthogonalize(np.zeros(shape), coeffs) == 0).all()


def test_cubic_coefficients_converge_to_the_polar_factor():
    u = np.random.default_rng(3).standard_normal((5, 8))
    got = M.orthogonalize(u, [(1.5, -0.5, 0.0)] * 40)
    assert np.allclose(got @ got.T, np.eye(5), atol=1e-12)


# ---- refusals, before any HIP call ----------------------------------------------

def _status(call):
    with pytest.raises(capi.FsdpError) as ei:
        call()
    return ei.value.status


def test_muon_calls_reject_unbound_and_bad_arguments_without_gpu():
    assert _status(lambda: capi.fsdp_muon_momentum(None, 0x1000, 0.9, stream=0)) == capi.FSDP_E_INVAL
    assert _status(lambda: capi.fsdp_muon_reduce_momentum(None, 0x1000, 0x2000, 0.9,
                                                          stream=0)) == capi.FSDP_E_INVAL
    assert _status(lambda: capi.fsdp_muon_update(None, 0x1000, 0x2000, 0.1, 0.0,
                                                 stream=0)) == capi.FSDP_E_INVAL
    p = capi.fsdp_plan_create([4, 3], [2, 1], 2, 0, 1)
    try:
        for call in (lambda: capi.fsdp_muon_momentum(p, 0x1000, 0.9, stream=0),
                     lambda: capi.fsdp_muon_reduce_momentum(p, 0x1000, 0x2000, 0.9, stream=0),
                     lambda: capi.fsdp_muon_update(p, 0x1000, 0x2000, 0.1, 0.0, stream=0)):
            assert _status(call) == capi.FSDP_E_STATE
    finally:
        capi.fsdp_plan_destroy(p)


def test_muon_binding_rejects_undersized_and_host_tensors():
    import torch
    p = capi.fsdp_plan_create([8, 3], [4, 1], 2, 0, 1)
    try:
        info = capi.fsdp_plan_info(p)
        n, S, k = info.world, info.S, info.n_params
        i16 = lambda m: torch.zeros(m, dtype=torch.int16)
        f32 = lambda m: torch.zeros(m, dtype=torch.float32)
        for call, make, need in (
                (lambda b: capi.fsdp_muon_momentum(p, b, 0.9, stream=0), i16, S),
                (lambda b: capi.fsdp_muon_reduce_momentum(p, b, 0x1000, 0.9, stream=0), i16, n * S),
                (lambda b: capi.fsdp_muon_reduce_momentum(p, 0x1000, b, 0.9, stream=0), i16, S),
                (lambda b: capi.fsdp_muon_update(p, b, 0x1000, 0.1, 0.0, stream=0), i16, S),
                (lambda b: capi.fsdp_muon_update(p, 0x1000, b, 0.1, 0.0, stream=0), i16, S),
                (lambda b: capi.fsdp_muon_update(p, 0x1000, 0x2000, 0.1, 0.0, scales=b, stream=0),
                 f32, k)):
            with pytest.raises(ValueError, match="bytes"):
                call(make(need - 1))
            with pytest.raises(ValueError, match="GPU tensor"):
                call(make(need))
    finally:
        capi.fsdp_plan_destroy(p)


def test_ortho_plan_layout_and_refusals():
    ns = [(3.4445, -4.7750, 2.0315)] * 5
    p = capi.fsdp_ortho_plan_create([5, 0, 300], [7, 4, 200], ns)
    n, ws = capi.fsdp_ortho_plan_info(p)
    assert n == 3 and ws > 0 and ws % 256 == 0
    assert _status(lambda: capi.fsdp_ortho_execute(p, 0x1000, ws, stream=0)) == capi.FSDP_E_STATE
    ptr = [0x10000, 0, 0x20000]
    out = [0x30000, 0, 0x40000]
    for ins, outs, dtype, status in (
            ([0, 0, 0x20000], out, 0, capi.FSDP_E_INVAL),
            (ptr, [0x30000, 0, 0], 0, capi.FSDP_E_INVAL),
            (ptr, out, 2, capi.FSDP_E_UNSUPPORTED),
            ([0x10001, 0, 0x20000], out, 0, capi.FSDP_E_ALIGN),
            ([0x10002, 0, 0x20000], out, 1, capi.FSDP_E_ALIGN),
            (ptr, [0x30000, 0, 0x40001], 0, capi.FSDP_E_ALIGN),
            (ptr, [0x30000, 0, 0x30000 + 2 * 34], 0, capi.FSDP_E_INVAL),
            (ptr, [0x20000, 0, 0x40000], 0, capi.FSDP_E_INVAL),
            (ptr, [0x30000, 0, 0x10000 + 2 * 34], 0, capi.FSDP_E_INVAL),
            ([0x10000, 0, 0x30000], [0x30000 + 59990 * 4, 0, 0x90000], 1, capi.FSDP_E_INVAL)):
        assert _status(lambda: capi.fsdp_ortho_bind(p, ins, outs, dtype, stream=0)) == status
    capi.fsdp_ortho_plan_destroy(p)
    capi.fsdp_ortho_plan_destroy(None)
    assert capi.fsdp_ortho_plan_info(capi.fsdp_ortho_plan_create([], [], ns))[1] == 0
    for rows, cols, coeffs, eps, status in (
            ([-1], [2], ns, 0.0, capi.FSDP_E_INVAL),
            ([2], [-1], ns, 0.0, capi.FSDP_E_INVAL),
            ([2], [2], [], 0.0, capi.FSDP_E_INVAL),
            ([2], [2], ns, -1.0, capi.FSDP_E_INVAL),
            ([2], [2], ns, float("nan"), capi.FSDP_E_INVAL),
            ([2], [2], [(float("inf"), 0, 0)], 0.0, capi.FSDP_E_INVAL),
            ([2], [2], [(float("nan"), 0, 0)], 0.0, capi.FSDP_E_INVAL),
            ([2], [2], ns * 13, 0.0, capi.FSDP_E_UNSUPPORTED),
            ([2], [2], [(4.5, 0, 0)], 0.0, capi.FSDP_E_UNSUPPORTED),
            ([2], [2], [(2.0, 0, 0)] * 3, 0.0, capi.FSDP_E_UNSUPPORTED),
            ([2], [2], [(30.0, -60.0, 31.0)], 0.0, capi.FSDP_E_UNSUPPORTED),
            ([(1 << 20) + 1], [2], ns, 0.0, capi.FSDP_E_UNSUPPORTED),
            ([1 << 17], [1 << 17], ns, 0.0, capi.FSDP_E_UNSUPPORTED)):
        assert _status(lambda: capi.fsdp_ortho_plan_create(rows, cols, coeffs, eps)) == status
    for call in (lambda: capi.fsdp_ortho_plan_info(None), lambda: capi.fsdp_ortho_bind(None, [], []),
                 lambda: capi.fsdp_ortho_bind(None, [], [], stream=0),
                 lambda: capi.fsdp_ortho_execute(None, 0, 0, stream=0)):
        with pytest.raises((capi.FsdpError, RuntimeError, AssertionError)):
            call()
    with pytest.raises(ValueError):
        capi.fsdp_ortho_plan_create([1], [1, 2], ns)
    with pytest.raises(ValueError):
        capi.fsdp_ortho_plan_create([1], [1], [(1.0, 2.0)])
