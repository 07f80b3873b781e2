"""8-bit matrices on the GPU: copy-in with block scales, quantising and restoring bit
for bit against the oracle, products and linear layers against fp64."""
import numpy as np
import pytest
import torch

from oracle import fsdp as O
from oracle import q8 as Q

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("sharded_shard_amd.capi")
from sharded_shard_amd import q8  # noqa: E402
from sharded_shard_amd.group import ShardedGroup  # noqa: E402

DEV = "cuda"
FMTS = ["e4m3", "e5m2"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def rng(*key):
    return np.random.default_rng([ord(c) for c in repr(key)])


def data(rows, cols, *key):
    """Rows of different size, columns that stand out."""
    g = rng(rows, cols, *key)
    x = g.standard_normal((rows, cols)) * np.exp(g.standard_normal((rows, 1)))
    return (x * (1 + 20 * (g.random(cols) < 0.02))).astype(np.float32)


def gpu(x, bf16):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return t.bfloat16() if bf16 else t


def host(t):
    return t.detach().double().cpu().numpy()


def same_codes(got, want, fmt, what=""):
    """Equal values, and NaN for NaN."""
    a, b = Q.decode(got, fmt), Q.decode(want, fmt)
    assert np.array_equal(a, b, equal_nan=True), (what, int((a != b).sum()))


def check_quantized(q, x, blocks, fmt):
    codes, lines = Q.quantize(x, blocks, fmt)
    assert np.array_equal(q.scales_view().cpu().numpy(), lines), "scales"
    same_codes(q.codes_view().cpu().numpy(), codes, fmt, "codes")


# ---- quantise and restore -----------------------------------------------------------

SIZES = [(1, 1), (1, 128), (2, 130), (7, 8), (127, 129), (128, 128), (129, 257), (300, 1000),
         (33, 4097), (4099, 24), (1100, 1400)]


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_quantize_matches_the_oracle(size, fmt, bf16):
    x = gpu(data(*size, fmt), bf16)
    h = host(x)
    for blocks in ("rows", "cols", "tiles"):
        check_quantized(q8.quantize(x, blocks, fmt), h, blocks, fmt)
    rows, cols = q8.quantize(x, "both", fmt)
    check_quantized(rows, h, "rows", fmt)
    check_quantized(cols, h, "cols", fmt)


def special(fmt):
    """Blocks at the borders: fmax 2^k and the next value, zeros, the smallest and largest
    numbers, scales under and over the one that the 16-bit path starts at."""
    top = Q.FORMATS[fmt][3]
    x = np.zeros((256, 384))
    g = rng("special", fmt)
    for i in range(256):
        x[i] = g.uniform(-1, 1, 384) * 2.0 ** (i % 250 - 126)
        x[i, 5] = top * 2.0 ** (i % 200 - 110)                  # exactly at the border
        if i % 3 == 0:
            x[i, 5] *= 1 + 2.0 ** -7                            # and past it
    x[10], x[:, 20], x[130:140, 128:256] = 0.0, 0.0, -0.0
    x[200:, 256:] *= 2.0 ** -60
    x[3, :128] = 2.0 ** -133 * g.integers(0, 100, 128)          # bf16's subnormals
    x[4, :128] = 3.3e38 * g.uniform(-1, 1, 128)
    return np.clip(x, -3.38e38, 3.38e38).astype(np.float32)


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_borders(fmt, bf16):
    x = gpu(special(fmt), bf16)
    h = host(x)
    for blocks in ("rows", "cols", "tiles"):
        check_quantized(q8.quantize(x, blocks, fmt), h, blocks, fmt)
    # columns whose scales lie at and around 2^(24 - 127)
    g = rng("low")
    y = (g.standard_normal((128, 128)) * 2.0 ** (np.arange(128) % 60 - 125)).astype(np.float32)
    y = gpu(y, bf16)
    check_quantized(q8.quantize(y, "cols", fmt), host(y), "cols", fmt)
    z = gpu((g.standard_normal((300, 128)) * 2.0 ** (np.arange(128) - 90.0)).astype(np.float32), bf16)
    check_quantized(q8.quantize(z, "cols", fmt), host(z), "cols", fmt)


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", [(200, 300), (1100, 1400)], ids=str)
def test_what_is_not_finite_shows_and_sets_no_scale(size, fmt, bf16):
    x = data(*size, "nan")
    x[5, 7], x[5, 8], x[60, 200], x[150, 150] = np.nan, np.inf, -np.inf, -np.nan
    x[70, :] = np.inf                       # nothing finite left in a row
    x[:, 90] = np.nan                       # or a column
    t = gpu(x, bf16)
    h = host(t)
    for blocks in ("rows", "cols", "tiles"):
        q = q8.quantize(t, blocks, fmt)
        check_quantized(q, h, blocks, fmt)
        back = host(q8.dequantize(q, torch.float32))
        assert np.isnan(back[:, 90]).all()
        keep = (np.arange(size[1]) != 90) & (np.arange(size[1]) != 7)
        assert (np.isinf(back[70, keep]) if fmt == "e5m2" else np.isnan(back[70, keep])).all()
    for q, blocks in zip(q8.quantize(t, "both", fmt), ("rows", "cols")):
        check_quantized(q, h, blocks, fmt)


def test_quantize_strides_and_what_lies_around():
    """x inside a wider matrix and at an odd element; codes and scales inside wider ones,
    whose other bytes stay."""
    for fmt, bf16, rows, cols, skip in (("e4m3", True, 150, 201, 1), ("e5m2", False, 129, 64, 3),
                                        ("e4m3", True, 1, 1, 0), ("e4m3", True, 200, 304, 8)):
        wide = gpu(data(rows, cols + 37, "wide"), bf16)
        x = wide[:, skip:skip + cols]
        h = host(x)
        for blocks in ("rows", "cols", "tiles"):
            lines, length = q8.scale_lines(rows, cols, blocks)
            for pad, at in ((11, 3), (16, 16)):
                codes = torch.full((rows, cols + 2 * pad), 0x5A, dtype=torch.uint8, device=DEV)
                scales = torch.full((lines, -(-length // 4) * 4 + 8), 0x5A, dtype=torch.uint8, device=DEV)
                q = q8.Q8(codes[:, at:at + cols], scales[:, 4:4 + length], blocks, fmt)
                q8.quantize(x, blocks, fmt, out=q)
                check_quantized(q, h, blocks, fmt)
                codes[:, at:at + cols] = 0x5A
                scales[:, 4:4 + length] = 0x5A
                assert (codes == 0x5A).all() and (scales == 0x5A).all()
                out = torch.full((rows, cols + 9), 7.0, dtype=torch.bfloat16, device=DEV)
                q8.quantize(x, blocks, fmt, out=q)
                q8.dequantize(q, out=out[:, 5:5 + cols])
                v = Q.values(*Q.quantize(h, blocks, fmt), blocks, fmt).astype(np.float32)
                assert np.array_equal(host(out[:, 5:5 + cols]), O.bf16_to_f32(O.bf16_rne(v)))
                assert (out[:, :5] == 7).all() and (out[:, 5 + cols:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blocks", ["rows", "cols", "tiles"])
@pytest.mark.parametrize("size", [(1, 5), (130, 200), (4097, 260), (1200, 2000)], ids=str)
def test_dequantize_matches_the_oracle(size, blocks, fmt):
    """Any code and any byte that does not leave fp32: exact in fp32, rounded once to bf16."""
    g = rng(size, blocks, fmt)
    q = q8.Q8.empty(size, blocks, fmt)
    codes = g.integers(0, 256, size, dtype=np.uint8)
    lines = g.integers(0, 230, q.scales_view().shape, dtype=np.uint8)
    lines.flat[0] = 255
    q.codes_view().copy_(torch.from_numpy(codes))
    q.scales_view().copy_(torch.from_numpy(lines))
    want = Q.values(codes, lines, blocks, fmt)
    got = host(q8.dequantize(q, torch.float32))
    assert np.array_equal(got, want, equal_nan=True)
    half = host(q8.dequantize(q))
    with np.errstate(all="ignore"):
        w = O.bf16_to_f32(O.bf16_rne(want.astype(np.float32))).astype(np.float64)
    assert np.array_equal(half, w, equal_nan=True)


def test_dequantize_a_per_parameter_scale():
    """The FP8 copy-in's weights: no blocks, a divisor; one more rounding."""
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(5).view(10, 128)
    s = torch.tensor([3.7], device=DEV)
    q = q8.Q8(codes, None, "tensor", divisor=s)
    want = (Q.decode(codes.cpu().numpy(), "e4m3").astype(np.float32) / np.float32(3.7))
    assert np.array_equal(q8.dequantize(q, torch.float32).cpu().numpy(), want, equal_nan=True)


# ---- products ------------------------------------------------------------------------

def held(rows, cols, blocks, fmt, *key):
    """A quantised matrix, on the GPU and in fp64."""
    q = q8.quantize(gpu(data(rows, cols, *key), True), blocks, fmt)
    return q, Q.values(q.codes_view().cpu().numpy(), q.scales_view().cpu().numpy(), blocks, fmt)


def check_product(got, a, b, what=""):
    g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    a, b = g(a), g(b)
    c, s = a @ b, a.abs() @ b.abs()
    k = a.shape[1]
    tol = 2.0 ** -8 * c.abs() + (1 + 2.0 ** -8) * s * (
        7 * 2.0 ** -13 + (k / 8 + k / 128 + 24) * 2.0 ** -24) + 2.0 ** -133
    bad = (got.double() - c).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def test_the_tolerance_is_the_oracles():
    a, b = rng("t").standard_normal((3, 200)), rng("u").standard_normal((200, 4))
    c = a @ b
    s = np.abs(a) @ np.abs(b)
    want = 2.0 ** -8 * np.abs(c) + (1 + 2.0 ** -8) * s * (
        7 * 2.0 ** -13 + (200 / 8 + 200 / 128 + 24) * 2.0 ** -24) + 2.0 ** -133
    assert np.allclose(Q.product_tolerance(a, b, c), want, rtol=1e-12)


# rows, columns, inner: every tile, its edges, few rows, long and short sums
MNK = [(1, 1, 1), (1, 64, 128), (3, 33, 47), (16, 1000, 256), (17, 9000, 130), (32, 129, 1024),
       (33, 64, 64), (64, 64, 128), (65, 63, 129), (100, 300, 515), (128, 128, 2048), (130, 250, 16),
       (256, 256, 8200), (257, 511, 300), (1000, 1500, 400), (2049, 2305, 272), (300, 5000, 1000),
       (5000, 300, 136)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mnk", MNK, ids=str)
def test_product_forms(mnk, fmt):
    m, n, k = mnk
    # x W^T, dy W, dy^T x
    for ta, tb in ((False, True), (False, False), (True, False)):
        ba = "cols" if ta else "rows"
        bb = "rows" if tb else "cols"
        a, av = held(*((k, m) if ta else (m, k)), ba, fmt, "a", fmt)
        for blocks in (bb, "tiles"):
            b, bv = held(*((n, k) if tb else (k, n)), blocks, "e4m3", "b", blocks)
            got = q8.product(a, b, ta, tb)
            assert got.shape == (m, n)
            check_product(got, av.T if ta else av, bv.T if tb else bv, (ta, tb, blocks))
            assert torch.equal(got, q8.product(a, b, ta, tb)), "the same bits every time"


@pytest.mark.parametrize("ta,tb", [(False, True), (False, False), (True, False)])
def test_product_goes_from_tile_to_tile(ta, tb):
    """More tiles of 256 than CUs, of sizes that end inside one."""
    m, n, k = 4300, 4500, 400
    a, av = held(*((k, m) if ta else (m, k)), "cols" if ta else "rows", "e4m3", "a")
    b, bv = held(*((n, k) if tb else (k, n)), "tiles", "e4m3", "b")
    check_product(q8.product(a, b, ta, tb), av.T if ta else av, bv.T if tb else bv)


@pytest.mark.parametrize("ta,tb", [(False, True), (False, False), (True, False)])
def test_product_of_tiles_with_tiles_and_of_tensors(ta, tb):
    m, n, k = 200, 300, 333
    a, av = held(*((k, m) if ta else (m, k)), "tiles", "e4m3", "a")
    g = rng("tensor", ta, tb)
    shape = (n, k) if tb else (k, n)
    codes = g.integers(0, 255, shape, dtype=np.uint8)
    codes[(codes & 127) == 127] = 0
    div = torch.tensor([2.5], device=DEV)
    for d in (None, div):
        b = q8.Q8(torch.from_numpy(codes).to(DEV), None, "tensor", "e4m3", divisor=d)
        bv = Q.decode(codes, "e4m3") / (1.0 if d is None else 2.5)
        check_product(q8.product(a, b, ta, tb), av.T if ta else av, bv.T if tb else bv, d)
    # few rows, and both divided (two roundings of the factor: inside the fp32 terms)
    if not ta and tb:
        x = q8.Q8(torch.from_numpy(codes[:5].copy()).to(DEV), None, "tensor", divisor=div)
        b = q8.Q8(torch.from_numpy(codes).to(DEV), None, "tensor", divisor=div)
        check_product(q8.product(x, b, ta, tb), Q.decode(codes[:5], "e4m3") / 2.5,
                      Q.decode(codes, "e4m3").T / 2.5)


@pytest.mark.parametrize("mnk", [(5, 200, 300), (150, 200, 300), (600, 700, 131)], ids=str)
@pytest.mark.parametrize("ta,tb", [(False, True), (False, False), (True, False)])
def test_product_reads_nothing_around_its_operands(mnk, ta, tb):
    """NaN codes before, between and after the rows, NaN bytes around the scales; the result
    inside a wider matrix whose other elements stay; addresses and strides of every kind."""
    m, n, k = mnk
    def inside(q, at, ld):
        rows, cols = q.shape
        flat = torch.full((at + rows * ld + 64,), 0x7F, dtype=torch.uint8, device=DEV)
        codes = flat[at:at + rows * ld].view(rows, ld)[:, :cols]
        codes.copy_(q.codes_view())
        lines, length = q.scales_view().shape
        pitch = -(-length // 4) * 4 + 4
        s = torch.full((lines + 2, pitch), 0xFF, dtype=torch.uint8, device=DEV)
        s[1:1 + lines, :length].copy_(q.scales_view())
        return q8.Q8(codes, s[1:1 + lines, :length], q.blocks, q.format)
    a, av = held(*((k, m) if ta else (m, k)), "cols" if ta else "rows", "e4m3", "a")
    b, bv = held(*((n, k) if tb else (k, n)), "rows" if tb else "cols", "e4m3", "b")
    for at, more in ((0, 0), (16, 16), (3, 5), (16, 1)):
        up = lambda c: -(-c // 16) * 16 + more
        x, w = inside(a, at, up(a.cols)), inside(b, at, up(b.cols))
        for ldo, first in ((n, 0), (n + 8, 8), (n + 3, 1)):
            out = torch.full((m + 1, ldo + first), 7.0, dtype=torch.bfloat16, device=DEV)
            view = out[:m, first:first + n]
            q8.product(x, w, ta, tb, out=view)
            check_product(view, av.T if ta else av, bv.T if tb else bv, (at, more, ldo, first))
            view.fill_(7.0)
            assert (out == 7).all()


def test_product_of_nothing():
    e = q8.Q8.empty
    for m, n, k, ta, tb in ((0, 5, 64, False, True), (5, 0, 64, False, False), (70, 90, 0, False, True),
                            (70, 90, 0, True, False), (3, 90, 0, False, True)):
        a = e((k, m) if ta else (m, k), "cols" if ta else "rows")
        b = e((n, k) if tb else (k, n), "tiles")
        out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device=DEV)
        assert (q8.product(a, b, ta, tb, out=out) == 0).all() and out.shape == (m, n)


@pytest.mark.parametrize("m", [4, 100, 300])
def test_nan_stays_in_its_row_and_column(m):
    n, k = 200, 300
    x = data(m, k, "x")
    x[2, 17] = np.nan
    a = q8.quantize(gpu(x, True), "rows")
    b, bv = held(n, k, "tiles", "e4m3", "b")
    got = q8.product(a, b, trans_b=True)
    assert torch.isnan(got[2]).all()
    keep = [i for i in range(m) if i != 2]
    av = Q.values(a.codes_view().cpu().numpy(), a.scales_view().cpu().numpy(), "rows", "e4m3")
    check_product(got[keep], av[keep], bv.T)
    # a scale of NaN: its block's rows
    a = q8.quantize(gpu(np.nan_to_num(x), True), "rows")
    a.scales_view()[1, 3] = 255
    got = q8.product(a, b, trans_b=True)
    assert torch.isnan(got[3]).all() and not torch.isnan(got[:3]).any()
    # an infinity in E5M2
    x[2, 17] = np.inf
    a = q8.quantize(gpu(x, True), "rows", "e5m2")
    got = q8.product(a, b, trans_b=True)
    assert not torch.isfinite(got[2]).any() and torch.isfinite(got[keep]).all()


def test_product_with_scales_at_the_ends():
    """2^-127 with large ones, and results past bf16's range."""
    codes = torch.full((64, 128), 0x38, dtype=torch.uint8, device=DEV)        # ones
    def of(byte):
        return q8.Q8(codes, torch.full((1, 64), byte, dtype=torch.uint8, device=DEV), "rows")
    for x, y in ((0, 127), (0, 254), (127, 127), (200, 40), (254, 120), (60, 60), (5, 120)):
        got = q8.product(of(x), of(y), trans_b=True)
        want = torch.full((64, 64), 128.0, dtype=torch.float64) * 2.0 ** (x + y - 254)
        assert torch.equal(got.cpu().double(), want.float().bfloat16().double()), (x, y)
    assert torch.isinf(q8.product(of(254), of(254), trans_b=True)).all()


def test_product_past_two_to_the_32():
    """Codes, and then results, that lie past 4 GiB."""
    m, k = (1 << 20) + 300, 4200
    a = q8.Q8.empty((m, k), "rows")
    block = held(512, k, "rows", "e4m3", "big")
    for i in range(0, m, 512):
        n = min(512, m - i)
        a.codes[i:i + n].copy_(block[0].codes[:n])
        a.scales[:, i:i + n].copy_(block[0].scales[:, :n])
    assert m * a.c.ld > 1 << 32
    b, bv = held(40, k, "tiles", "e4m3", "b")
    got = q8.product(a, b, trans_b=True)
    last = (m - 512) // 512 * 512
    for i in (0, last, last + 512):
        n = min(512, m - i)
        check_product(got[i:i + n], block[1][:n], bv.T, i)
    del a, got
    m, n, k = (1 << 20) + 300, 2200, 64
    a = q8.quantize(gpu(data(m, k, "rows"), True), "rows")
    b, bv = held(n, k, "tiles", "e4m3", "b")
    got = q8.product(a, b, trans_b=True)
    assert got.numel() * 2 > 1 << 32
    av = Q.values(a.codes[-400:].cpu().numpy(), a.scales[:, -400:].cpu().numpy(), "rows", "e4m3")
    check_product(got[-400:], av, bv.T)
    back = q8.quantize(got, "cols")
    x = host(got[-(m % 128):])
    same_codes(back.codes[-(m % 128):].cpu().numpy(), Q.quantize(x, "cols", "e4m3")[0], "e4m3")


# ---- streams and graphs ---------------------------------------------------------------

def test_on_another_stream():
    m, n, k = 300, 256, 640
    x = gpu(data(m, k, "x"), True)
    b, bv = held(n, k, "tiles", "e4m3", "b")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for how in (st, st.cuda_stream):
        a = q8.quantize(x, "rows", stream=how)
        got = q8.product(a, b, trans_b=True, stream=how)
        back = q8.dequantize(a, torch.float32, stream=how)
        st.synchronize()
        check_product(got, host(back), bv.T)


def test_captured_steps_replay():
    """Two graphs of a layer's steps with memory of their own, replayed in turn with eager
    work between, on inputs that change."""
    t, n, k = 200, 320, 8200
    w, _ = held(n, k, "tiles", "e4m3", "w")
    xs = [gpu(data(t, k, i), True) for i in range(3)]
    dys = [gpu(data(t, n, "dy", i), True) for i in range(3)]
    def steps(x, dy, dw):
        layer = q8.Linear8(w)
        y = layer.forward(x)
        return y, layer.backward(dy, dw), dw
    graphs = []
    for i in range(2):
        x, dy = xs[i].clone(), dys[i].clone()
        dw = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            steps(x, dy, dw)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = steps(x, dy, dw)
        graphs.append((g, x, dy, outs))
    for turn in range(6):
        g, x, dy, outs = graphs[turn % 2]
        x.copy_(xs[turn % 3])
        dy.copy_(dys[(turn + 1) % 3])
        g.replay()
        want = steps(x, dy, torch.empty(n, k, dtype=torch.bfloat16, device=DEV))
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), turn


# ---- linear layers -----------------------------------------------------------------------

@pytest.mark.parametrize("tokens", [1, 20, 333, 0, 1024])
@pytest.mark.parametrize("fmt", FMTS)
def test_linear_is_its_parts(tokens, fmt):
    n, k = 260, 515
    w, _ = held(n, k, "tiles", "e4m3", "w")
    for bf16 in (True, False):
        x, dy = gpu(data(tokens, k, "x"), bf16), gpu(data(tokens, n, "dy"), bf16)
        layer = q8.Linear8(w, grad_format=fmt)
        y = layer.forward(x)
        (saved,) = layer.saved
        dw = torch.full((n, k), 7, dtype=torch.int16, device=DEV)
        dx = layer.backward(dy, dw)
        assert not layer.saved
        xr, xc = q8.quantize(x, "both")
        dr, dc = q8.quantize(dy, "both", fmt)
        assert torch.equal(saved.codes, xc.codes) and torch.equal(saved.scales, xc.scales)
        assert torch.equal(y, q8.product(xr, w, trans_b=True))
        assert torch.equal(dx, q8.product(dr, w))
        assert torch.equal(dw.view(torch.bfloat16), q8.product(dc, xc, trans_a=True))


def test_linear_without_some():
    n, k, t = 128, 256, 70
    w, _ = held(n, k, "tiles", "e4m3", "w")
    x, dy = gpu(data(t, k, "x"), True), gpu(data(t, n, "dy"), True)
    layer = q8.Linear8(w)
    y = layer.forward(x)
    assert torch.equal(layer.forward(x, save=False), y) and len(layer.saved) == 1
    dw = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    dx = layer.backward(dy, dw)
    layer.forward(x)
    assert torch.equal(layer.backward(dy, None), dx)
    layer.forward(x)
    only = torch.empty_like(dw)
    assert layer.backward(dy, only, need_input=False) is None and torch.equal(only, dw)
    layer.forward(x)
    assert layer.backward(dy, None, need_input=False) is None
    with pytest.raises(RuntimeError):
        layer.backward(dy, dw)


def test_linear_keeps_microbatches_in_order():
    n, k = 128, 256
    w, _ = held(n, k, "tiles", "e4m3", "w")
    layer, alone = q8.Linear8(w), q8.Linear8(w)
    xs, dys = [gpu(data(64 + i, k, i), True) for i in range(3)], [gpu(data(64 + i, n, i), True) for i in range(3)]
    for x in xs:
        layer.forward(x)
    a, b = (torch.empty(n, k, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for x, dy in zip(xs, dys):
        dx = layer.backward(dy, a)
        alone.forward(x)
        assert torch.equal(dx, alone.backward(dy, b)) and torch.equal(a, b)


def test_linear_gradients_are_the_formulas_and_the_differences():
    """On small whole numbers the 8-bit values are the numbers, and sums of under 2^8 are
    exact in bf16: y = x W^T, and the gradients equal the differences."""
    g = rng("whole")
    t, n, k = 128, 128, 128
    def whole(rows, cols, share):
        x = g.integers(-1, 2, (rows, cols)) * (g.random((rows, cols)) < share)
        return x.astype(np.float32)
    x, w, dy = whole(t, k, 0.3), whole(n, k, 0.3), whole(t, n, 0.3)
    wq = q8.quantize(gpu(w, True), "tiles")
    assert np.array_equal(host(q8.dequantize(wq, torch.float32)), w)
    loss = lambda xx: float((host(q8.Linear8(wq).forward(gpu(xx, True))) * dy).sum())
    layer = q8.Linear8(wq)
    y = layer.forward(gpu(x, True))
    assert np.array_equal(host(y), x.astype(np.float64) @ w.T)
    dw = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    dx = host(layer.backward(gpu(dy, True), dw))
    assert np.array_equal(dx, dy.astype(np.float64) @ w)
    assert np.array_equal(host(dw), dy.T.astype(np.float64) @ x)
    for i, j in ((0, 0), (5, 77), (127, 127), (64, 1)):
        step = np.zeros_like(x)
        step[i, j] = 1.0
        assert loss(x + step) - loss(x - step) == 2 * dx[i, j]
        up, down = (q8.quantize(gpu(w + s * step[:n], True), "tiles") for s in (1, -1))
        of = lambda q: float((host(q8.Linear8(q).forward(gpu(x, True))) * dy).sum())
        assert of(up) - of(down) == 2 * host(dw)[i, j]


def test_linear_backward_on_another_stream():
    n, k, t = 256, 512, 300
    w, _ = held(n, k, "tiles", "e4m3", "w")
    x, dy = gpu(data(t, k, "x"), True), gpu(data(t, n, "dy"), True)
    one, two = q8.Linear8(w), q8.Linear8(w)
    a, b = (torch.empty(n, k, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    one.forward(x)
    dx = one.backward(dy, a)
    two.forward(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for how in (st, st.cuda_stream):
        got = two.backward(dy, b, stream=how)
        st.synchronize()
        assert torch.equal(got, dx) and torch.equal(a, b)
        two.forward(x)
        torch.cuda.synchronize()


# ---- copy-in -----------------------------------------------------------------------------

CASES = [
    ("probe", [(32, 16), (32,), (4, 32), (4,)], 2),
    ("one", [(1, 1)], 1),
    ("ragged-n6", [(1000, 70), (333,), (77, 129), (1, 2048), (1,), (64, 2048)], 6),
    ("empty", [(5, 3), (0, 4), (7,), (1, 5), (13, 2)], 4),
    ("tiles", [(300, 1000), (4096, 33), (70001,)], 8),
    ("odd-n12", [(1000, 37), (4097,), (129, 3), (25, 8)], 12),
    ("aligned-n8", [(1024, 256), (2048, 512)], 8),
    ("wide", [(3, 70001), (200, 300)], 2),
]


def two_d(shape):
    return shape[0], int(np.prod(shape[1:], dtype=np.int64)) if len(shape) > 1 else 1


@pytest.mark.parametrize("align", [1, 8])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_copy_in_with_block_scales(case, align):
    """Every rank's bytes, their maximum, every rank's segment, the gathered matrices: those of
    the full matrix quantised in one piece; and nothing written around."""
    name, shapes, world = case
    full = []
    for i, s in enumerate(shapes):
        g = rng(name, i)
        x = g.standard_normal(two_d(s)) * 2.0 ** g.integers(-12, 12, (two_d(s)[0], 1))
        full.append(x.astype(np.float32))
    if full[0].size > 3:
        full[0].flat[1], full[0].flat[2] = np.nan, -np.inf
        full[-1][...] = 0 if name == "empty" else full[-1]
    groups, bytes_ = [], []
    for r in range(world):
        g = ShardedGroup(shapes, world, r, align)
        for i, e in enumerate(g.entries):
            g.shard_view(g.master_flat, i).copy_(
                torch.from_numpy(full[i][e.row_begin:e.row_begin + e.local_rows].reshape(-1).copy()))
        buf = torch.full((g.n_block_scales + 64,), 0x5A, dtype=torch.uint8, device=DEV)
        g.block_scales(buf[32:32 + g.n_block_scales])
        got = buf.cpu().numpy()
        assert (got[:32] == 0x5A).all() and (got[32 + g.n_block_scales:] == 0x5A).all()
        at, want = 0, []
        for i, (x, e) in enumerate(zip(full, g.entries)):
            rows, cols = x.shape
            b = np.zeros((-(-rows // 128), -(-cols // 128)), np.uint8)
            if e.local_rows:
                part = Q.block_bytes(x[e.row_begin:e.row_begin + e.local_rows], "tiles", "e4m3",
                                     e.row_begin % 128)
                b[e.row_begin // 128:e.row_begin // 128 + len(part)] = part
            want.append(b.reshape(-1))
        assert np.array_equal(got[32:32 + g.n_block_scales], np.concatenate(want)), r
        groups.append(g)
        bytes_.append(buf[32:32 + g.n_block_scales].clone())
    scales = torch.stack(bytes_).amax(0)
    S = groups[0].S
    ag = torch.full((world * S + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    for r, g in enumerate(groups):
        g.pack_fp8_blocks(ag[32 + r * S:32 + (r + 1) * S], scales)
        seg = ag[32 + r * S:32 + (r + 1) * S].cpu().numpy()
        for i, e in enumerate(g.entries):
            codes, _ = Q.quantize(full[i], "tiles", "e4m3")
            mine = codes[e.row_begin:e.row_begin + e.local_rows].reshape(-1)
            same_codes(seg[e.shard_offset:e.shard_offset + e.valid_numel], mine, "e4m3", (r, i))
            assert (seg[e.shard_offset + e.valid_numel:e.shard_offset + e.seg_numel] == 0).all()
    assert (ag[:32] == 0x5A).all() and (ag[32 + world * S:] == 0x5A).all()
    g = groups[0]
    g.bind_full_fp8()
    g.unpack_fp8(ag[32:32 + world * S])
    for i, x in enumerate(full):
        q = g.full_q8(i, scales)
        codes, lines = Q.quantize(x, "tiles", "e4m3")
        same_codes(q.codes_view().cpu().numpy(), codes, "e4m3")
        assert np.array_equal(q.scales_view().cpu().numpy().reshape(-1), lines.reshape(-1))
        assert np.array_equal(host(q8.dequantize(q, torch.float32)),
                              Q.values(codes, lines, "tiles", "e4m3"), equal_nan=True)
    for g in groups:
        g.close()


def test_copy_in_saturates_and_takes_any_byte():
    g = ShardedGroup([(130, 40)], 1, 0)
    x = data(130, 40, "sat")
    x[0, :5] = [np.inf, -np.inf, np.nan, 3e38, -3e38]
    g.master_flat[:130 * 40].copy_(torch.from_numpy(x.reshape(-1)))
    seg = torch.empty(g.S, dtype=torch.uint8, device=DEV)
    for byte in (0, 1, 60, 120, 127, 200, 253, 254, 255):
        scales = torch.tensor([byte, 127], dtype=torch.uint8, device=DEV)
        g.pack_fp8_blocks(seg, scales)
        s = np.where(np.arange(130) < 128, np.nan if byte == 255 else 2.0 ** (byte - 127.0), 1.0)
        want = Q.encode(x.astype(np.float64) / s[:, None], "e4m3", saturate=True)
        same_codes(seg.cpu().numpy().reshape(130, 40), want, "e4m3", byte)
    g.close()


def test_copy_in_refuses_overlap_and_small_buffers():
    g = ShardedGroup([(130, 40)], 1, 0)
    raw = g.master_flat.view(torch.uint8)
    ok = torch.empty(g.S, dtype=torch.uint8, device=DEV)
    scales = torch.empty(2, dtype=torch.uint8, device=DEV)
    for call in (lambda: g.block_scales(raw), lambda: g.pack_fp8_blocks(raw, scales),
                 lambda: g.pack_fp8_blocks(ok, ok[5:])):
        with pytest.raises(capi.FsdpError) as e:
            call()
        assert e.value.status == capi.FSDP_E_INVAL
    for call in (lambda: g.block_scales(scales[:1]), lambda: g.pack_fp8_blocks(ok[1:], scales),
                 lambda: g.block_scales(scales.cpu())):
        with pytest.raises(ValueError):
            call()
    g.close()


# ---- together -----------------------------------------------------------------------------

def test_a_training_step_in_8_bits():
    """Two ranks, one after the other: block scales and their maximum, copy-in, copy-out, the
    layer's steps on each rank's tokens, the gradients' reduction and the update."""
    n, k, t, world = 300, 200, 90, 2
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    w = data(n, k, "w") * 0.02
    groups = [ShardedGroup([(n, k)], world, r, 8) for r in range(world)]
    S = groups[0].S
    scales = torch.zeros(groups[0].n_block_scales, dtype=torch.uint8, device=DEV)
    for g in groups:
        e = g.entries[0]
        g.shard_view(g.master_flat, 0).copy_(
            torch.from_numpy(w[e.row_begin:e.row_begin + e.local_rows].reshape(-1).copy()))
        mine = torch.empty_like(scales)
        g.block_scales(mine)
        scales = torch.maximum(scales, mine)
    ag = torch.empty(world * S, dtype=torch.uint8, device=DEV)
    for r, g in enumerate(groups):
        g.pack_fp8_blocks(ag[r * S:(r + 1) * S], scales)
    codes, lines = Q.quantize(w, "tiles", "e4m3")
    wv = Q.values(codes, lines, "tiles", "e4m3")
    rs = torch.empty(world, world * S, dtype=torch.int16, device=DEV)
    for r, g in enumerate(groups):
        g.bind_full_fp8()
        g.unpack_fp8(ag)
        g.bind_full_grad()
        layer = q8.Linear8(g.full_q8(0, scales), grad_format="e5m2")
        x, dy = gpu(data(t, k, "x", r), True), gpu(data(t, n, "dy", r) * 1e-3, True)
        xr = Q.values(*Q.quantize(host(x), "rows", "e4m3"), "rows", "e4m3")
        check_product(layer.forward(x), xr, wv.T)
        dx = layer.backward(dy, g.full_grad_view(0))
        dr = Q.values(*Q.quantize(host(dy), "rows", "e5m2"), "rows", "e5m2")
        check_product(dx, dr, wv)
        dc = Q.values(*Q.quantize(host(dy), "cols", "e5m2"), "cols", "e5m2")
        xc = Q.values(*Q.quantize(host(x), "cols", "e4m3"), "cols", "e4m3")
        check_product(g.full_grad_view(0).view(torch.bfloat16), dc.T, xc)
        g.pack_reduce_scatter(rs[r])
    p = O.plan([(n, k)], world, 0, 8)
    for r, g in enumerate(groups):
        rows = torch.cat([rs[j, r * S:(r + 1) * S] for j in range(world)])
        before = [g.shard_view(g.master_flat, 0).cpu().numpy().copy()]
        g.reduce(rows)
        g.adamw(1, **hp)
        p = O.plan([(n, k)], world, r, 8)
        grads = O.reduce(p, rows.cpu().numpy().view(np.uint16).reshape(world, S))
        m, v = [np.zeros_like(before[0])], [np.zeros_like(before[0])]
        O.adamw(before[0], grads[0], m[0], v[0], 1, **hp)
        assert np.array_equal(g.shard_view(g.master_flat, 0).cpu().numpy(), before[0])
        g.close()


# ---- what Python refuses ---------------------------------------------------------------------

def test_python_refusals():
    x = gpu(data(40, 64, "x"), True)
    q = q8.quantize(x, "rows")
    w = q8.quantize(gpu(data(32, 64, "w"), True), "tiles")
    bad = [lambda: q8.quantize(x.cpu()), lambda: q8.quantize(x[0]), lambda: q8.quantize(x.double()),
           lambda: q8.quantize(x.t()), lambda: q8.quantize(x, "columns"), lambda: q8.quantize(x, "rows", "e3m4"),
           lambda: q8.quantize(x, "cols", out=q), lambda: q8.quantize(x[:5], "rows", out=q),
           lambda: q8.quantize(x[:1].expand(5, 64)), lambda: q8.dequantize(q, torch.float16),
           lambda: q8.dequantize(q, out=torch.empty(40, 63, dtype=torch.bfloat16, device=DEV)),
           lambda: q8.product(q, w, trans_b=True, out=torch.empty(40, 32, device=DEV)),
           lambda: q8.product(q, w, trans_b=True, out=torch.empty(39, 32, dtype=torch.bfloat16, device=DEV)),
           lambda: q8.Q8(q.codes, None, "rows"), lambda: q8.Q8(q.codes, q.scales[:, :39], "rows"),
           lambda: q8.Q8(q.codes, q.scales, "rows", divisor=torch.ones(2, device=DEV)),
           lambda: q8.Linear8(q), lambda: q8.Linear8(w, "e3m4"),
           lambda: q8.Linear8(q8.quantize(x, "tiles", "e5m2")), lambda: q8.Linear8(w).forward(x[:, :63])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for f in (lambda: q8.product(q, w), lambda: q8.product(q, w, True, True),
              lambda: q8.product(q8.quantize(x, "cols"), w, trans_b=True),
              lambda: q8.product(q, q8.quantize(x, "tiles", "e5m2"), trans_b=True)):
        with pytest.raises(capi.FsdpError):
            f()


def test_injected_fault_reaches_the_caller(monkeypatch):
    x = gpu(data(40, 64, "x"), True)
    w = q8.quantize(gpu(data(32, 64, "w"), True), "tiles")
    layer = q8.Linear8(w)
    monkeypatch.setenv("FSDP_FAULT", "launch@2")
    with pytest.raises(capi.FsdpError) as e:
        layer.forward(x)                                # the product's launch
    assert e.value.status == capi.FSDP_E_HIP and not layer.saved
    monkeypatch.delenv("FSDP_FAULT")
    layer.forward(x)
    assert len(layer.saved) == 1
