"""Orthogonalisation on the GPU against the fp64 iterate of the oracle.

Tolerance.  The output is bf16: half a step, 2^-8 of the value at most, which
over a matrix is at most 2^-8 in the relative 2-norm.  The products round X, A
and B to fp16, half a step 2^-11 each; an iteration's slope at a singular value
in [0.7, 1.2], a + 3 b s^2 + 5 c s^4, is at most 3.4 in size, and what the
rounding of A, of B and of X puts into an iteration is at most |b| s^2 + 2 |c|
s^4, 2 (|b| s^2 + |c| s^4) and |b s^2 + c s^4| half steps, about 10 of 2^-11
at s = 1 in the worst case and a third of that where they do not all add up:
2^-8 once more.  Up to 128 rows every operand has a second fp16 part, 2^-22, of
which the iterations magnify at most 485 times (3.4445^5): 2^-13, for each of
four roundings: 2^-11 in place of the second 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import fsdp as O
from oracle import muon as M

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("sharded_shard_amd.capi")
from sharded_shard_amd.group import NS_COEFFS, Orthogonalizer, ShardedGroup  # noqa: E402

DEV = "cuda"
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def matrix(shape, seed, kind="noise", dtype=torch.bfloat16):
    """CPU matrix: white noise, a falling spectrum, or low rank."""
    g = torch.Generator().manual_seed(seed)
    r, c = shape
    k = max(1, min(shape) // 8)
    if kind == "noise":
        x = torch.randn(r, c, generator=g)
    elif kind == "falling":
        x = torch.randn(r, k, generator=g) / torch.arange(1, k + 1) @ torch.randn(k, c, generator=g)
        x = x + 0.05 * torch.randn(r, c, generator=g)
    else:
        x = torch.randn(r, 2, generator=g) @ torch.randn(2, c, generator=g)
    return (1e-3 * x).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def run(mats, coeffs=NS_COEFFS, eps=1e-7, outs=None):
    """Outputs of one execution over CPU matrices, in guarded memory."""
    ins = [m.to(DEV) for m in mats]
    guard = 64
    bufs = [torch.full((m.numel() + 2 * guard,), 7.0, dtype=torch.bfloat16, device=DEV) for m in mats]
    outs = [b[guard:guard + m.numel()].view(m.shape) for b, m in zip(bufs, mats)]
    with Orthogonalizer([m.shape for m in mats], coeffs, eps) as o:
        o.bind(ins, outs)
        o.allocate(torch.full((max(1, o.workspace_bytes),), 0xFF, dtype=torch.uint8, device=DEV))
        o.execute()
        torch.cuda.synchronize()
    for b, i, m in zip(bufs, ins, mats):
        assert (b[:guard] == 7).all() and (b[guard + m.numel():] == 7).all(), "write outside"
        assert torch.equal(i.cpu().view(torch.int16), m.view(torch.int16)), "input changed"
    return outs


def close(got, u, coeffs=NS_COEFFS, eps=1e-7):
    inner = 2.0 ** -11 if min(u.shape) <= 128 else HALF
    want = M.orthogonalize(f64(u), coeffs, eps)
    got = f64(got)
    assert np.isfinite(got).all()
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= (HALF + inner) * norm, (u.shape, err / norm)
    rms = norm / np.sqrt(want.size)
    assert (np.abs(got - want) <= HALF * np.abs(want) + 10 * inner * rms).all(), u.shape


SHAPES = [(1, 1), (1, 7), (9, 1), (4, 32), (32, 16), (33, 31), (64, 64), (65, 2047), (127, 128),
          (128, 129), (129, 128), (200, 130), (130, 515), (256, 256), (257, 255), (384, 1000),
          (1000, 384), (1, 2048), (2048, 5), (640, 640), (31, 1024), (32, 1025), (2100, 20),
          (50, 512), (513, 33), (1300, 64), (97, 128), (100, 129), (1000, 128), (128, 500)]


@pytest.mark.parametrize("kind", ["noise", "falling", "low"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_matches_the_fp64_iterate(shape, kind):
    u = matrix(shape, hash(shape) % 1000, kind)
    close(run([u])[0], u)


@pytest.mark.parametrize("shape", [(5, 3), (40, 300), (200, 333), (333, 200)],
                         ids=lambda s: "%dx%d" % s)
def test_fp32_inputs(shape):
    u = matrix(shape, 3, "falling", torch.float32)
    close(run([u])[0], u)


def test_many_matrices_in_one_plan_repeat_and_are_as_right_as_each_alone():
    """The same plan gives the same bits; alone, a matrix's sums may be split
    otherwise, which moves fp32 sums and what is rounded from them."""
    shapes = [(200, 300), (1, 5), (0, 4), (300, 200), (64, 64), (130, 700), (200, 300)]
    mats = [matrix(s, i, "falling") for i, s in enumerate(shapes)]
    together = run(mats)
    again = run(mats)
    for u, x, y in zip(mats, together, again):
        assert torch.equal(x, y)
        if u.numel():
            close(x, u)
            close(run([u])[0], u)


@pytest.mark.parametrize("shape", [(8, 20), (150, 260), (260, 150)], ids=lambda s: "%dx%d" % s)
def test_in_place_and_misaligned_memory(shape):
    u = matrix(shape, 1)
    want = run([u])[0]
    n = u.numel()
    for off in (0, 1, 3):
        buf = torch.zeros(n + 8, dtype=torch.bfloat16, device=DEV)
        x = buf[off:off + n].view(shape)
        x.copy_(u)
        with Orthogonalizer([shape]) as o:
            o.bind([x])
            o.execute()
            torch.cuda.synchronize()
        assert torch.equal(x, want), off
        assert (buf[:off] == 0).all() and (buf[off + n:] == 0).all()


@pytest.mark.parametrize("shape", [(6, 9), (150, 200), (200, 150)], ids=lambda s: "%dx%d" % s)
def test_special_matrices(shape):
    """Zeros stay zeros; a NaN or an infinity spreads over its matrix and no
    further; the largest and smallest norms lose nothing."""
    z = torch.zeros(shape, dtype=torch.bfloat16)
    u = matrix(shape, 2)
    bad = [u.clone() for _ in range(3)]
    bad[0][shape[0] // 2, 1] = float("nan")
    bad[1][0, shape[1] - 1] = float("inf")
    bad[2][shape[0] - 1, 0] = float("-inf")
    outs = run([z, bad[0], u, bad[1], z, bad[2]])
    assert (outs[0] == 0).all() and (outs[4] == 0).all()
    for k in (1, 3, 5):
        assert torch.isnan(outs[k]).all()
    close(outs[2], u)
    for scale in (2.0 ** 120, 2.0 ** -100, 2.0 ** -30, 2.0 ** -13):
        v = (u.double() * scale).to(torch.bfloat16)
        for eps in (0.0, 1e-7):
            close(run([v], eps=eps)[0], v, eps=eps)
    assert torch.isnan(run([z], eps=0.0)[0]).all()


@pytest.mark.parametrize("coeffs", [((1.5, -0.5, 0.0),) * 3, ((2.0, -1.5, 0.5),),
                                    ((3.4445, -4.775, 2.0315),) * 2 + ((1.5, -0.5, 0.0),) * 7,
                                    ((1.0, 0.0, 0.0),), ((0.0, 1.0, -0.25),) * 2], ids=range(5))
@pytest.mark.parametrize("shape", [(30, 50), (260, 180)], ids=lambda s: "%dx%d" % s)
def test_other_coefficients(coeffs, shape):
    u = matrix(shape, 4, "noise")
    close(run([u], coeffs)[0], u, coeffs)


def test_long_sum_and_offsets():
    """Few rows of many columns, both ways round."""
    for shape in ((130, 40000), (40000, 130), (3, 100001), (100, 20000), (20000, 60)):
        u = matrix(shape, 5, "noise")
        close(run([u])[0], u)


@pytest.mark.parametrize("tall", [False, True])
def test_more_than_2_to_31_elements(tall):
    """U = [V V .. V], k times: X X^T is V's, so the result is V's over sqrt(k), here
    16.  Both sides are within the tolerance of the exact one."""
    v = matrix((2100, 4096), 4, "falling")
    want = run([v])[0].float()
    k, n = 256, 2100 * 4096 * 256
    assert n > 2 ** 31
    u = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    d = v.to(DEV)
    if tall:
        d, want = d.t().contiguous(), want.t().contiguous()
        u.view(k, 4096, 2100).copy_(d)
    else:
        u.view(2100, k, 4096).copy_(d[:, None])
    out = torch.zeros_like(u)
    with Orthogonalizer([(4096 * k, 2100) if tall else (2100, 4096 * k)]) as o:
        o.bind([u], [out])
        o.execute()
        torch.cuda.synchronize()
    norm = want.norm().item()
    for i in range(k):
        x = out.view(k, 4096, 2100)[i] if tall else out.view(2100, k, 4096)[:, i]
        assert (x.float() * 16 - want).norm().item() <= 4 * HALF * norm, i


# counts at which a plan takes other tiles for its products: X X^T and A A in
# 128, 192 and 256, B X in 128, 192 and 256 with its term a X before and along
# the sum, X X^T in parts
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape,count", [((139, 140), 60), ((1040, 1037), 12), ((677, 680), 40),
                                         ((257, 260), 60), ((440, 523), 40), ((797, 800), 16),
                                         ((900, 7900), 2)], ids=str)
def test_every_tile_with_edges(shape, count, dtype):
    """One wide and one tall matrix, the others of the plan copies of them: equal
    shapes and inputs give equal bits."""
    r, c = shape
    us = [matrix(shape, 11, "falling", dtype), matrix((c, r), 12, "noise", dtype)]
    ins = [u.to(DEV) for u in us] * (count // 2)
    outs = [torch.full(u.shape, 7.0, dtype=torch.bfloat16, device=DEV) for u in ins]
    with Orthogonalizer([u.shape for u in ins]) as o:
        o.bind(ins, outs)
        o.allocate(torch.full((o.workspace_bytes,), 0xFF, dtype=torch.uint8, device=DEV))
        o.execute()
        torch.cuda.synchronize()
    for u, x in zip(us, outs):
        close(x, u)
    for i, x in enumerate(outs):
        assert torch.equal(x, outs[i % 2]), i


def test_captured_execution_replays_like_an_eager_one():
    shapes = [(150, 260), (20, 30), (260, 150)]
    mats = [matrix(s, i, "falling").to(DEV) for i, s in enumerate(shapes)]
    eager = [torch.empty_like(m) for m in mats]
    outs = [torch.empty_like(m) for m in mats]
    a, b = Orthogonalizer(shapes), Orthogonalizer(shapes)
    a.bind(mats, eager)
    b.bind(mats, outs)
    a.allocate()
    b.allocate()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.execute(stream=side)
    for k in range(3):
        for m in mats:
            m.mul_(1.5).add_(1e-4)
        a.execute()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager, outs):
            assert torch.equal(x, y), k
    del graph
    a.close()
    b.close()


def test_two_executions_at_once_with_their_own_workspaces():
    shape = (300, 500)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    mats = [matrix(shape, i, "falling").to(DEV) for i in range(2)]
    outs = [torch.empty_like(m) for m in mats]
    plans = [Orthogonalizer([shape]) for _ in mats]
    for p, m, o in zip(plans, mats, outs):
        p.bind([m], [o])
        p.allocate()
    torch.cuda.synchronize()
    for _ in range(4):
        for p, s in zip(plans, streams):
            p.execute(stream=s)
    torch.cuda.synchronize()
    for m, o in zip(mats, outs):
        assert torch.equal(o, run([m.cpu()])[0])


def test_refusals_on_the_device():
    u = matrix((130, 2), 0).to(DEV).repeat(1, 80).contiguous()
    n = u.numel()
    o = Orthogonalizer([u.shape, u.shape])
    x = torch.zeros(4 * n, dtype=torch.bfloat16, device=DEV)
    views = lambda a, b: [x[a:a + n].view(u.shape), x[b:b + n].view(u.shape)]

    def refused(status, call):
        with pytest.raises(capi.FsdpError) as ei:
            call()
        assert ei.value.status == status, str(ei.value)

    refused(capi.FSDP_E_STATE, lambda: o.execute())
    refused(capi.FSDP_E_INVAL, lambda: o.bind([u, u], views(0, n - 1)))
    refused(capi.FSDP_E_INVAL, lambda: o.bind(views(0, n), views(64, 3 * n)))
    with pytest.raises(ValueError):
        o.bind([u], [u])
    with pytest.raises(ValueError):
        o.bind([u, u.float()], views(0, n))
    with pytest.raises(ValueError):
        o.bind([u, u.t().contiguous().t()], views(0, n))
    o.bind([u, u], views(0, n))         # the same input twice
    need = o.workspace_bytes
    ws = torch.empty(need + 512, dtype=torch.uint8, device=DEV)
    refused(capi.FSDP_E_INVAL, lambda: capi.fsdp_ortho_execute(o.plan, ws.data_ptr(), need - 1))
    refused(capi.FSDP_E_INVAL, lambda: capi.fsdp_ortho_execute(o.plan, 0, need))
    refused(capi.FSDP_E_ALIGN, lambda: capi.fsdp_ortho_execute(o.plan, ws.data_ptr() + 8, need))
    with pytest.raises(ValueError):
        o.allocate(ws[:need - 1])
    o.execute()
    torch.cuda.synchronize()
    assert torch.equal(x[:n], x[n:2 * n])
    with Orthogonalizer([(1, 2000)]) as over:     # the workspace holds the input
        big = torch.empty(over.workspace_bytes + 8192, dtype=torch.uint8, device=DEV)
        over.bind([big[512:4512].view(torch.bfloat16).view(1, 2000)])
        refused(capi.FSDP_E_INVAL, lambda: capi.fsdp_ortho_execute(over.plan, big))
    o.close()


@pytest.mark.parametrize("as_handle", [False, True])
def test_first_execution_on_another_stream_takes_memory_of_that_stream(as_handle):
    """A block that torch freed on its current stream may still be in use there."""
    u = matrix((300, 500), 1).to(DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with Orthogonalizer([(300, 500)]) as o:
        o.bind([u], [torch.empty_like(u)])
        torch.cuda.empty_cache()
        freed = torch.empty(o.workspace_bytes, dtype=torch.uint8, device=DEV)
        was = freed.data_ptr()
        del freed
        o.execute(stream=s.cuda_stream if as_handle else s)
        assert o.workspace.data_ptr() != was
        torch.cuda.synchronize()
        first = o._bound[1][0].clone()
        o.execute()
        torch.cuda.synchronize()
        assert torch.equal(first, o._bound[1][0])


def test_parameters_of_a_group_from_any_iterable():
    g = ShardedGroup([(8, 16), (12, 4)], 1, 0, optimizer="muon")
    with g.orthogonalizer(i for i in (1, 0)) as o:
        assert o.shapes == [(12, 4), (8, 16)]
        o.execute()
        torch.cuda.synchronize()
    with pytest.raises(capi.FsdpError) as ei:        # the same matrix twice
        g.orthogonalizer([0, 0])
    assert ei.value.status == capi.FSDP_E_INVAL
    g.close()


def test_injected_launch_fault_reaches_the_caller(monkeypatch):
    u = matrix((8, 16), 0).to(DEV)
    with Orthogonalizer([(8, 16)]) as o:
        o.bind([u])
        monkeypatch.setenv("FSDP_FAULT", "launch")
        with pytest.raises(capi.FsdpError, match="injected") as ei:
            o.execute()
        assert ei.value.status == capi.FSDP_E_HIP
        monkeypatch.delenv("FSDP_FAULT")
        o.execute()
        torch.cuda.synchronize()


# ---- the whole step --------------------------------------------------------------

@pytest.mark.parametrize("owned", [False, True], ids=["every-rank", "owned"])
@pytest.mark.parametrize("n,shapes", [(1, [(20, 30)]), (2, [(32, 16), (4, 32)]),
                                      (3, [(50, 70), (1, 9), (70, 50), (140, 150)])])
def test_whole_step_over_all_ranks(n, shapes, owned):
    """Momentum, all-gather of the updates, orthogonalisation, the way back and
    the update, two steps on every rank of the group (the collectives are
    copies between the ranks' buffers here)."""
    mu, lr, wd = 0.9, 0.05, 0.1
    gs = [ShardedGroup(shapes, n, r, optimizer="muon") for r in range(n)]
    S = gs[0].S
    rng = np.random.default_rng(n)
    plans = [O.plan(shapes, n, r) for r in range(n)]
    masters = [[rng.standard_normal(e.valid_numel).astype(np.float32) for e in p.entries] for p in plans]
    ms = [[np.zeros(e.valid_numel, np.float32) for e in p.entries] for p in plans]
    for g, xs in zip(gs, masters):
        for i, x in enumerate(xs):
            g.shard_view(g.master_flat, i).copy_(torch.from_numpy(x.copy()))
    scales = np.array([max(1.0, r / c) ** 0.5 for r, c in shapes], np.float32)
    sc = torch.from_numpy(scales).to(DEV)
    # a matrix on every rank, or each on one: rank i % n has matrix i
    mine = [[i for i in range(len(shapes)) if not owned or i % n == r] for r in range(n)]
    orth = [g.orthogonalizer(k) for g, k in zip(gs, mine)]
    ag = torch.zeros(n, S, dtype=torch.int16, device=DEV)
    params = torch.zeros(n, S, dtype=torch.int16, device=DEV)
    for step in range(2):
        rs = [O.bf16_rne(rng.standard_normal((n, S)).astype(np.float32)) for _ in range(n)]
        for r, g in enumerate(gs):
            g.muon_reduce_momentum(torch.from_numpy(rs[r].reshape(-1).view(np.int16)).to(DEV), ag[r], mu)
        for g, o in zip(gs, orth):
            g.unpack(ag.view(-1))
            o.execute()
        want = np.stack([M.reduce_momentum(p, x, m, mu, True) for p, x, m in zip(plans, rs, ms)])
        assert np.array_equal(ag.cpu().numpy().view(np.uint16), want)
        full = [O.bf16_to_f32(u).reshape(s) for u, s in zip(O.unpack(plans[0], want), shapes)]
        for i, u in enumerate(full):
            close(gs[i % n].full_view(i).view(torch.bfloat16), torch.from_numpy(np.array(u)))
        # the oracle goes on from the GPU's orthogonalised matrices
        outs = [gs[i % n].full_view(i).cpu().numpy().view(np.uint16) for i in range(len(shapes))]
        for r, (g, p) in enumerate(zip(gs, plans)):
            parts = [o.reshape(-1)[e.row_begin * e.cols:e.row_begin * e.cols + e.valid_numel]
                     for o, e in zip(outs, p.entries)]
            seg = None
            if owned:
                host = np.zeros(S, np.uint16)
                for e, o in zip(p.entries, parts):
                    host[e.shard_offset:e.shard_offset + e.valid_numel] = o
                seg = torch.from_numpy(host.view(np.int16)).to(DEV)
            g.muon_update(seg, params[r], lr, wd, scales=sc)
            want = M.update(p, masters[r], parts, scales, lr, wd)
            assert np.array_equal(params[r].cpu().numpy().view(np.uint16), want)
            for i, x in enumerate(masters[r]):
                got = g.shard_view(g.master_flat, i).cpu().numpy()
                assert np.array_equal(got.view(np.uint32), x.view(np.uint32))
    for o in orth:
        o.close()
    for g in gs:
        g.close()
