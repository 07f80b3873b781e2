"""The Muon momentum and update on the GPU, bit for bit against the oracle
(both round every fp32 operation once, in the same order)."""
import numpy as np
import pytest
import torch

from oracle import fsdp as O
from oracle import muon as M
from workloads import synth

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("sharded_shard_amd.capi")
from sharded_shard_amd.group import ShardedGroup  # noqa: E402

DEV = "cuda"
GUARD = 512

CASES = [
    ("probe", [(32, 16), (4, 32)], 2, (0, 1)),
    ("one", [(1, 1)], 1, (0,)),
    ("ragged-n6", [(1000, 70), (77, 129), (1, 2048), (64, 2048)], 6, (0, 1, 5)),
    ("empty", [(5, 3), (0, 4), (1, 5), (13, 2)], 4, (0, 3)),
    ("tiles", [(300, 1000), (4096, 33), (129, 257)], 8, (0, 7)),
    ("odd-n12", [(1000, 37), (129, 3), (25, 8)], 12, (0, 11)),
    ("aligned-n8", [(1024, 256), (64, 512)], 8, (3,)),
    ("wide-n64", [(5000, 24), (64, 72), (129, 8), (1, 8)], 64, (0, 43)),
]
IDS = [c[0] for c in CASES]
MU, LR, WD = 0.95, 0.02, 0.1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def u16(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def f32(t):
    return t.detach().cpu().contiguous().numpy()


def same(got, want, what):
    """Equal bits, NaNs of any payload alike."""
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    assert np.array_equal(got[~nan].view(np.uint32), want[~nan].view(np.uint32)), what


def same_bf16(got, want, what):
    same(O.bf16_to_f32(got), O.bf16_to_f32(want), what)


def guarded(n):
    buf = torch.full((n + 2 * GUARD,), 0x5A5A, dtype=torch.int16, device=DEV)
    return buf, buf[GUARD:GUARD + n]


def untouched(buf, n):
    h = u16(buf)
    assert (h[:GUARD] == 0x5A5A).all() and (h[GUARD + n:] == 0x5A5A).all()


def fill(g, flat, key, std=1.0):
    """The group's shards filled; returns host copies."""
    out = []
    for i, e in enumerate(g.entries):
        x = synth.normal_f32(e.valid_numel, std, key + (i,))
        g.shard_view(flat, i).copy_(x)
        out.append(x.numpy().copy())
    return out


def host(g, flat):
    return [f32(g.shard_view(flat, i)) for i in range(len(g.entries))]


def rows(n, S, key):
    return synth.bf16_bits_to_u16(synth.normal_bf16_bits(n * S, 1e-3, key)).reshape(n, S)


def dev(u):
    return torch.from_numpy(np.ascontiguousarray(u).reshape(-1).view(np.int16)).to(DEV)


@pytest.mark.parametrize("align", [1, 8])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_momentum_matches_oracle(case, nesterov, align):
    name, shapes, n, ranks = case
    for r in ranks:
        g = ShardedGroup(shapes, n, r, align, optimizer="muon")
        p = O.plan(shapes, n, r, align)
        ms = [np.zeros(e.valid_numel, np.float32) for e in g.entries]
        buf, seg = guarded(g.S)
        for step in range(2):
            gs = fill(g, g.grad_flat, (name, r, step))
            g.muon_momentum(seg, MU, nesterov)
            want = M.momentum(p, gs, ms, MU, nesterov)
            same_bf16(u16(seg), want, "segment")
            for got, m in zip(host(g, g.m_flat), ms):
                same(got, m, "m")
        untouched(buf, g.S)
        g.close()


@pytest.mark.parametrize("align", [1, 8])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_reduce_momentum_matches_oracle_and_the_two_calls(case, nesterov, align):
    name, shapes, n, ranks = case
    for r in ranks:
        a = ShardedGroup(shapes, n, r, align, optimizer="muon")
        b = ShardedGroup(shapes, n, r, align, optimizer="muon")
        p = O.plan(shapes, n, r, align)
        ms = fill(a, a.m_flat, (name, r))
        b.m_flat.copy_(a.m_flat)
        rs = rows(n, a.S, (name, "rs", r))
        for phase in (0, 1):         # the rows 16-byte aligned, and 2 bytes past
            d = torch.zeros(n * a.S + 8, dtype=torch.int16, device=DEV)[phase:phase + n * a.S]
            d.copy_(dev(rs))
            buf, seg = guarded(a.S)
            a.muon_reduce_momentum(d, seg, MU, nesterov)
            want = M.reduce_momentum(p, rs, ms, MU, nesterov)
            same_bf16(u16(seg), want, "segment")
            for got, m in zip(host(a, a.m_flat), ms):
                same(got, m, "m")
            untouched(buf, a.S)
            two = torch.empty_like(seg)
            b.reduce(d)
            b.muon_momentum(two, MU, nesterov)
            assert torch.equal(two, seg) and torch.equal(a.m_flat, b.m_flat)
        a.close()
        b.close()


@pytest.mark.parametrize("align", [1, 8])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_update_matches_oracle_from_segment_and_from_rows(case, align):
    name, shapes, n, ranks = case
    for r in ranks:
        g = ShardedGroup(shapes, n, r, align, optimizer="muon")
        p = O.plan(shapes, n, r, align)
        xs = fill(g, g.master_flat, (name, r), 0.02)
        full = [synth.bf16_bits_to_u16(synth.normal_bf16_bits(a * b, 0.02, (name, "o", i)))
                for i, (a, b) in enumerate(shapes)]
        mine, seg_u = [], np.full(p.S, 0x7FC0, np.uint16)     # NaN padding: never read
        for o, e in zip(full, p.entries):
            mine.append(o[e.row_begin * e.cols:e.row_begin * e.cols + e.valid_numel])
            seg_u[e.shard_offset:e.shard_offset + e.valid_numel] = mine[-1]
        for i, o in enumerate(full):
            if o.size:
                g.full_view(i).copy_(dev(o).view(g.rows[i], g.cols[i]))
        scales = np.linspace(0.5, 2.0, len(shapes)).astype(np.float32)
        sc = torch.from_numpy(scales).to(DEV)
        for src, s, out in (("segment", sc, True), ("rows", sc, True), ("rows", None, True),
                            ("segment", sc, False)):
            buf, seg = guarded(g.S)
            g.muon_update(dev(seg_u) if src == "segment" else None, seg if out else None, LR, WD,
                          scales=s)
            want = M.update(p, xs, mine, scales if s is not None else np.ones(len(shapes)), LR, WD)
            for got, x in zip(host(g, g.master_flat), xs):
                same(got, x, (src, "master"))
            if out:
                same_bf16(u16(seg), want, (src, "segment"))
            untouched(buf, g.S)
        g.close()


@pytest.mark.parametrize("op", ["momentum", "reduce", "update"])
def test_special_values_match_oracle(op):
    """NaN, infinities, zeros of both signs, subnormals and the largest values."""
    vals = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-40, 3.4e38, -3.4e38, 1.0],
                    np.float32)
    shapes, n, r = [(41, 25), (3, 7)], 3, 1
    g = ShardedGroup(shapes, n, r, optimizer="muon")
    p = O.plan(shapes, n, r)
    rng = np.random.default_rng(5)
    pick = lambda k: vals[rng.integers(0, len(vals), k)]
    state = [pick(e.valid_numel) for e in g.entries]
    flat = g.master_flat if op == "update" else g.m_flat
    for i, x in enumerate(state):
        g.shard_view(flat, i).copy_(torch.from_numpy(x.copy()))
    seg = torch.empty(g.S, dtype=torch.int16, device=DEV)
    if op == "momentum":
        gs = [pick(e.valid_numel) for e in g.entries]
        for i, x in enumerate(gs):
            g.shard_view(g.grad_flat, i).copy_(torch.from_numpy(x.copy()))
        g.muon_momentum(seg, MU, True)
        want = M.momentum(p, gs, state, MU, True)
    elif op == "reduce":
        rs = O.bf16_rne(pick(n * g.S)).reshape(n, g.S)
        g.muon_reduce_momentum(dev(rs), seg, MU, True)
        with np.errstate(all="ignore"):
            want = M.reduce_momentum(p, rs, state, MU, True)
    else:
        o = O.bf16_rne(pick(g.S))
        g.muon_update(dev(o), seg, LR, WD)
        mine = [o[e.shard_offset:e.shard_offset + e.valid_numel] for e in p.entries]
        want = M.update(p, state, mine, [1.0, 1.0], LR, WD)
    same_bf16(u16(seg), want, "segment")
    for got, x in zip(host(g, flat), state):
        same(got, x, "state")
    g.close()


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_shards_at_every_phase_and_mixed_ones(shift):
    """Shards at every 4-byte phase of 16, the gradient's phase the same or another."""
    shapes, n, r = [(97, 13), (1031, 1), (5, 8)], 3, 1
    p = O.plan(shapes, n, r, 1)
    for other in (shift, (shift + 1) % 4):
        g = ShardedGroup(shapes, n, r, optimizer="muon", bind=False)
        g.allocate()
        views, hosts = {}, {}
        for role, ph in (("master", shift), ("grad", other), ("m", shift)):
            base = torch.zeros(sum(e.valid_numel + 8 for e in g.entries) + 64, device=DEV)
            o, vs, hs = ph, [], []
            for i, e in enumerate(g.entries):
                x = synth.normal_f32(e.valid_numel, 1.0, (role, shift, i))
                v = base[o:o + e.valid_numel]
                v.copy_(x)
                vs.append(v)
                hs.append(x.numpy().copy())
                o += (e.valid_numel + 7) // 4 * 4
            views[role], hosts[role] = vs, hs
        capi.fsdp_bind(g.plan, views["master"], views["grad"], views["m"])
        seg = torch.empty(g.S, dtype=torch.int16, device=DEV)
        g.muon_momentum(seg, MU)
        same_bf16(u16(seg), M.momentum(p, hosts["grad"], hosts["m"], MU, True), "momentum")
        rs = rows(n, g.S, ("phase", shift))
        g.muon_reduce_momentum(dev(rs), seg, MU)
        same_bf16(u16(seg), M.reduce_momentum(p, rs, hosts["m"], MU, True), "reduce")
        o = rows(1, g.S, ("phase-o", shift))[0]
        g.muon_update(dev(o), seg, LR, WD)
        mine = [o[e.shard_offset:e.shard_offset + e.valid_numel] for e in p.entries]
        same_bf16(u16(seg), M.update(p, hosts["master"], mine, [1.0] * 3, LR, WD), "update")
        for role in ("master", "m"):
            for v, h in zip(views[role], hosts[role]):
                same(f32(v), h, role)
        g.close()


def test_refusals_leave_the_state_alone():
    shapes, n, r = [(8, 16)], 2, 0
    g = ShardedGroup(shapes, n, r, optimizer="muon")
    fill(g, g.master_flat, ("refuse",))
    was = g.master_flat.clone()
    seg = torch.zeros(2 * g.S, dtype=torch.int16, device=DEV)
    rs = torch.zeros(n * g.S, dtype=torch.int16, device=DEV)
    master16 = g.master_flat.view(torch.int16)
    m16 = g.m_flat.view(torch.int16)
    E = capi
    odd = seg.data_ptr() + 1
    for status, call in (
            (E.FSDP_E_INVAL, lambda: g.muon_momentum(seg, 1.0)),
            (E.FSDP_E_INVAL, lambda: g.muon_momentum(seg, float("nan"))),
            (E.FSDP_E_INVAL, lambda: g.muon_momentum(0, 0.9)),
            (E.FSDP_E_ALIGN, lambda: g.muon_momentum(odd, 0.9)),
            (E.FSDP_E_INVAL, lambda: g.muon_momentum(m16, 0.9)),
            (E.FSDP_E_INVAL, lambda: g.muon_reduce_momentum(rs, rs[g.S:], 0.9)),
            (E.FSDP_E_INVAL, lambda: g.muon_reduce_momentum(rs, m16, 0.9)),
            (E.FSDP_E_INVAL, lambda: g.muon_reduce_momentum(0, seg, 0.9)),
            (E.FSDP_E_INVAL, lambda: g.muon_update(seg, seg[g.S // 2:], 0.1, 0.0)),
            (E.FSDP_E_INVAL, lambda: g.muon_update(seg, master16, 0.1, 0.0)),
            (E.FSDP_E_INVAL, lambda: g.muon_update(None, g.full_flat, 0.1, 0.0)),
            (E.FSDP_E_INVAL, lambda: g.muon_update(seg, None, float("inf"), 0.0)),
            (E.FSDP_E_ALIGN, lambda: g.muon_update(seg, None, 0.1, 0.0, scales=odd)),
            (E.FSDP_E_INVAL, lambda: g.muon_update(seg, None, 0.1, 0.0, scales=g.master_flat)),
            (E.FSDP_E_ALIGN, lambda: g.muon_update(odd, None, 0.1, 0.0))):
        with pytest.raises(capi.FsdpError) as ei:
            call()
        assert ei.value.status == status, str(ei.value)
    torch.cuda.synchronize()
    assert torch.equal(g.master_flat, was) and not g.m_flat.any()
    with pytest.raises(ValueError):
        ShardedGroup(shapes, n, r, optimizer="sgd")
    with pytest.raises(capi.FsdpError):        # no exp_avg_sq: AdamW is refused
        g.adamw(1, 1e-3, 0.9, 0.999, 1e-8, 0.0)
    empty = ShardedGroup([(0, 4)], 2, 0, optimizer="muon")
    none = torch.empty(0, dtype=torch.int16, device=DEV)
    empty.muon_momentum(none, 0.9)
    empty.muon_reduce_momentum(none, none, 0.9)
    empty.muon_update(none, none, 0.1, 0.0)
    g.close()
    empty.close()


def test_captured_calls_replay_like_eager_ones_on_another_stream():
    shapes, n, r = CASES[2][1], 6, 5
    a, b = (ShardedGroup(shapes, n, r, optimizer="muon") for _ in range(2))
    for flat in ("m_flat", "master_flat"):
        fill(a, getattr(a, flat), ("graph", flat))
        getattr(b, flat).copy_(getattr(a, flat))
    rs = dev(rows(n, a.S, ("graph-rs",)))
    o = dev(rows(1, a.S, ("graph-o",)))
    segs = [torch.zeros(2, a.S, dtype=torch.int16, device=DEV) for _ in range(2)]

    def step(g, seg, stream=None):
        g.muon_reduce_momentum(rs, seg[0], MU, stream=stream)
        g.muon_update(o, seg[1], LR, WD, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(b, segs[1], side)
    for _ in range(3):
        step(a, segs[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(segs[0], segs[1])
        assert torch.equal(a.m_flat, b.m_flat) and torch.equal(a.master_flat, b.master_flat)
        rs.add_(0)
    del graph
    a.close()
    b.close()
