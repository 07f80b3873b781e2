"""Host-side checks of the 8-bit matrices: the oracle's pins, where block scales lie,
and the library's refusals (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import fsdp as O
from oracle import q8 as Q
from conftest import read_golden

capi = pytest.importorskip("sharded_shard_amd.capi")
from sharded_shard_amd import q8  # noqa: E402


# ---- the oracle against what it does not use ------------------------------------

def test_decode_matches_the_formats_definitions():
    c = np.arange(256, dtype=np.uint8)
    for fmt, t in (("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)):
        want = torch.from_numpy(c).view(t).double().numpy()
        assert np.array_equal(Q.decode(c, fmt), want, equal_nan=True)
    assert np.nanmax(Q.decode(c, "e4m3")) == 448.0
    assert Q.decode(np.uint8([1]), "e4m3")[0] == 2.0 ** -9
    v = Q.decode(c, "e5m2")
    assert np.max(v[np.isfinite(v)]) == 57344.0 and Q.decode(np.uint8([1]), "e5m2")[0] == 2.0 ** -16


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_encode_is_the_nearest_code_by_brute_force(fmt):
    rng = np.random.default_rng(5)
    v = Q.decode(np.arange(128), fmt)
    v = v[np.isfinite(v)]
    mid = (v[1:] + v[:-1]) / 2                     # the ties
    x = np.concatenate([v, mid, mid * (1 + 2.0 ** -40), mid * (1 - 2.0 ** -40),
                        rng.uniform(0, v[-1], 500), 2.0 ** rng.uniform(-20, 8, 500)])
    for sign in (1.0, -1.0):
        got = Q.encode(sign * x, fmt)
        d = np.abs(v[None, :] - x[:, None])
        best = d.min(1)
        near = Q.decode(got, fmt) * sign
        assert (np.abs(near - x) == best).all()
        tied = (d == best[:, None]).sum(1) > 1
        assert (got[tied] % 2 == 0).all()


def test_encode_agrees_with_the_copy_ins_oracle():
    x = np.random.default_rng(1).uniform(-460, 460, 4000).astype(np.float32)
    assert np.array_equal(Q.encode(x, "e4m3", saturate=True), O.e4m3_sat(x))


@pytest.mark.parametrize("fmt,top", [("e4m3", 448.0), ("e5m2", 57344.0)])
def test_scale_is_the_smallest_power_of_two(fmt, top):
    a = np.concatenate([2.0 ** np.arange(-140, 127, 1.0), top * 2.0 ** np.arange(-130, 100, 1.0),
                        np.nextafter(np.float32(top), np.float32(np.inf)) * 2.0 ** np.arange(-100, 100, 1.0)])
    b = Q.scale_byte(a, fmt).astype(np.float64)
    assert (a <= top * 2.0 ** (b - 127)).all()
    assert ((b == 0) | (a > top * 2.0 ** (b - 128))).all()
    assert Q.scale_byte(np.array([0.0]), fmt)[0] == 0


@pytest.mark.parametrize("blocks", ["rows", "cols", "tiles"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_is_off_by_half_a_step(blocks, fmt):
    """A normal code is off by at most half of 2^-3 (2^-2) of its value, which |x| bounds
    after the rounding; a subnormal one by half of the least, 2^-9 (2^-16) of its scale, and
    a block's scale is at most 2 amax / fmax."""
    x = np.random.default_rng(3).standard_normal((150, 300)) * np.exp(
        np.random.default_rng(4).standard_normal((150, 1)))
    codes, lines = Q.quantize(x, blocks, fmt)
    b = Q._spread(lines.T if blocks == "rows" else lines, blocks, 150, 300)
    s = 2.0 ** (b.astype(np.float64) - 127)
    mbits, least = (3, 2.0 ** -9) if fmt == "e4m3" else (2, 2.0 ** -16)
    err = np.abs(Q.values(codes, lines, blocks, fmt) - x)
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -(mbits + 1), s * least / 2)).all()


# ---- where block scales lie -------------------------------------------------------

SHAPES = [(300, 130), (0, 4), (1, 5), (129, 257), (7, 1)]


def test_plan_block_scales():
    plan = capi.fsdp_plan_create([s[0] for s in SHAPES], [s[1] for s in SHAPES], 3, 1)
    at = 0
    for i, (r, c) in enumerate(SHAPES):
        off, total = capi.fsdp_plan_block_scales(plan, i)
        assert off == at
        at += -(-r // 128) * -(-c // 128)
    assert total == at
    for bad in (-1, len(SHAPES)):
        with pytest.raises(capi.FsdpError) as e:
            capi.fsdp_plan_block_scales(plan, bad)
        assert e.value.status == capi.FSDP_E_INVAL
    capi.fsdp_plan_destroy(plan)
    empty = capi.fsdp_plan_create([], [], 2, 0)
    assert capi.fsdp_plan_block_scales(empty, 0) == (0, 0)
    capi.fsdp_plan_destroy(empty)


def test_scale_lines():
    assert q8.scale_lines(130, 300, "rows") == (3, 130)
    assert q8.scale_lines(130, 300, "cols") == (2, 300)
    assert q8.scale_lines(130, 300, "tiles") == (2, 3)
    assert q8.scale_lines(130, 300, "tensor") == q8.scale_lines(0, 300, "rows") == (0, 0)


# ---- refusals, before any HIP call --------------------------------------------------

BASE = 1 << 20      # addresses that no refused call reads


def mat(_rows, _cols, kind="rows", fmt="e4m3", /, at=BASE, **over):
    rows, cols = _rows, _cols
    blocks = kind
    lines, length = q8.scale_lines(rows, cols, blocks)
    ld = -(-cols // 16) * 16
    m = capi.Q8Struct(at, at + rows * ld, 0, rows, cols, ld, -(-length // 16) * 16,
                      q8.FORMATS[fmt], q8.BLOCKS[kind])
    for k, v in over.items():
        setattr(m, k, v)
    return m


def status(f, *args):
    with pytest.raises(capi.FsdpError) as e:
        f(*args, 0)             # the default stream
    return e.value.status


X = 1 << 30
OUT = 1 << 31


def quant(a, b=None, x=X, dtype=0, ldx=300):
    return status(capi.fsdp_q8_quantize, x, dtype, ldx, a, b)


def test_quantize_refusals():
    I, U, A = capi.FSDP_E_INVAL, capi.FSDP_E_UNSUPPORTED, capi.FSDP_E_ALIGN
    good = lambda **k: mat(200, 300, **k)
    assert quant(good(codes=0)) == I
    assert quant(good(scales=0)) == I
    assert quant(good(), x=0) == I
    assert quant(good(rows=-1)) == I
    assert quant(good(ld=299)) == I
    assert quant(good(pitch=196)) == I
    assert quant(good(), ldx=299) == I
    assert quant(good(divisor=BASE)) == I
    assert quant(good(rows=(1 << 22) + 1)) == U
    assert quant(good(ld=(1 << 22) + 16)) == U
    assert quant(good(format=2)) == U
    assert quant(good(blocks=4)) == U
    assert quant(good(blocks=0)) == U
    assert quant(good(), dtype=2) == U
    assert quant(good(), x=X + 1) == A
    assert quant(good(), x=X + 2, dtype=1) == A
    assert quant(good(scales=BASE + 200 * 304 + 2)) == A
    assert quant(good(pitch=202)) == A
    assert quant(good(divisor=BASE + 2)) == A
    # two outputs
    other = lambda **k: mat(200, 300, "cols", at=1 << 25, **k)
    assert quant(good(), other(format=1)) == I
    assert quant(good(), other(cols=299)) == I
    assert quant(good(), mat(200, 300, "rows", at=1 << 25)) == U
    assert quant(good(), mat(200, 300, "tiles", at=1 << 25)) == U
    assert quant(good(), mat(200, 300, "cols")) == I                # the same memory
    assert quant(good(), x=BASE + 200 * 304 - 2) == I               # x over the codes' end
    assert quant(good(scales=BASE + 4)) == I                        # scales among the codes


def test_dequantize_refusals():
    f = lambda q, out=OUT, dtype=0, ldo=300: status(capi.fsdp_q8_dequantize, q, out, dtype, ldo)
    assert f(mat(200, 300), out=0) == capi.FSDP_E_INVAL
    assert f(mat(200, 300), ldo=299) == capi.FSDP_E_INVAL
    assert f(mat(200, 300), dtype=7) == capi.FSDP_E_UNSUPPORTED
    assert f(mat(200, 300), out=OUT + 1) == capi.FSDP_E_ALIGN
    assert f(mat(200, 300), out=BASE) == capi.FSDP_E_INVAL
    assert f(mat(200, 300, divisor=OUT)) == capi.FSDP_E_INVAL


def prod(a, ta, b, tb, out=OUT, ldo=512, ws=1 << 34, n=1 << 33):
    return status(capi.fsdp_q8_product, a, ta, b, tb, out, ldo, ws, n)


def test_product_refusals():
    I, U, A = capi.FSDP_E_INVAL, capi.FSDP_E_UNSUPPORTED, capi.FSDP_E_ALIGN
    a, w = mat(200, 300), mat(400, 300, "tiles", at=1 << 25)
    assert prod(a, 0, w, 1, out=0) == I
    assert prod(a, 0, w, 1, ldo=399) == I
    assert prod(a, 0, w, 1, out=OUT + 1) == A
    assert prod(a, 2, w, 1) == I
    assert prod(a, 1, w, 1) == U
    assert prod(a, 0, w, 0) == I                                    # 300 against 400
    assert prod(mat(200, 300, "cols"), 0, w, 1) == U                # blocks across the sum
    assert prod(mat(300, 200, "rows"), 1, mat(300, 64, "cols", at=1 << 25), 0) == U
    assert prod(a, 0, mat(300, 64, "rows", at=1 << 25), 0) == U
    assert prod(a, 0, mat(400, 300, "cols", at=1 << 25), 1) == U
    assert prod(a, 0, mat(400, 300, "tiles", "e5m2", at=1 << 25), 1) == U
    assert prod(a, 0, w, 1, out=BASE) == I
    assert prod(a, 0, w, 1, out=w.scales - w.scales % 2) == I
    # an operand at an odd address is copied into a workspace first
    odd = mat(200, 300, codes=BASE + 1)
    assert prod(odd, 0, w, 1, ws=0) == I
    assert prod(odd, 0, w, 1, n=16) == I
    assert prod(odd, 0, w, 1, ws=(1 << 34) + 16) == A
    assert prod(odd, 0, w, 1, ws=BASE + 256) == I
    assert status(lambda *x: capi.fsdp_q8_product_workspace(*x[:-1]), a, 1, w, 1) == U


def test_product_workspace():
    w = mat(4096, 4096, "tiles", at=1 << 25)
    ws = capi.fsdp_q8_product_workspace
    assert ws(mat(4096, 4096), 0, w, 1) == 0                        # fills the CUs by itself
    copied = 200 * 4096
    assert ws(mat(200, 4096, ld=4097), 0, w, 1) - ws(mat(200, 4096), 0, w, 1) == copied
    assert ws(mat(200, 0), 0, mat(64, 0, "tiles"), 1) == 0
    assert ws(mat(0, 300), 0, mat(64, 300, "tiles"), 1) >= 0
    # a long sum of few results is cut into stretches
    assert ws(mat(8192, 256, "cols"), 1, mat(8192, 256, "cols"), 0) % (256 * 256 * 4) == 0


def fwd(w, x=X, dtype=0, ldx=300, tokens=64, saved=None, y=OUT, ldy=400, ws=1 << 34, n=1 << 33):
    return status(capi.fsdp_q8_linear_forward, w, x, dtype, ldx, tokens, saved, y, ldy, ws, n)


def bwd(w, saved, dy=X, dtype=0, lddy=400, fmt=0, dx=OUT, lddx=300, dw=1 << 33, lddw=300, ws=1 << 34,
        n=1 << 33):
    return status(capi.fsdp_q8_linear_backward, w, saved, dy, dtype, lddy, fmt, dx, lddx, dw, lddw, ws, n)


def test_linear_refusals():
    I, U, A = capi.FSDP_E_INVAL, capi.FSDP_E_UNSUPPORTED, capi.FSDP_E_ALIGN
    w, s = mat(400, 300, "tiles", at=1 << 25), mat(64, 300, "cols")
    assert fwd(mat(400, 300, "rows", at=1 << 25)) == U
    assert fwd(mat(400, 300, "tiles", "e5m2", at=1 << 25)) == U
    assert fwd(w, tokens=-1) == I
    assert fwd(w, tokens=(1 << 22) + 1) == U
    assert fwd(w, x=0) == I
    assert fwd(w, ldx=299) == I
    assert fwd(w, ldy=399) == I
    assert fwd(w, y=OUT + 1) == A
    assert fwd(w, saved=mat(64, 300, "rows")) == U
    assert fwd(w, saved=mat(63, 300, "cols")) == I
    assert fwd(w, saved=mat(64, 300, "cols", "e5m2")) == U
    assert fwd(w, n=100) == I
    assert fwd(w, ws=0) == I
    assert fwd(w, ws=(1 << 34) + 128) == A
    assert fwd(w, y=X) == I
    assert fwd(w, saved=mat(64, 300, "cols", at=OUT)) == I
    assert fwd(w, ws=1 << 25) == I
    assert bwd(w, mat(64, 300, "rows")) == U
    assert bwd(w, mat(64, 299, "cols")) == I
    assert bwd(w, s, fmt=2) == U
    assert bwd(w, s, dy=0) == I
    assert bwd(w, s, lddy=399) == I
    assert bwd(w, s, lddx=299) == I
    assert bwd(w, s, lddw=299) == I
    assert bwd(w, s, dx=OUT, dw=OUT) == I
    assert bwd(w, s, dw=BASE) == I
    assert bwd(w, s, n=0) == I
    with pytest.raises(capi.FsdpError) as e:
        capi.fsdp_q8_linear_workspace(mat(400, 300, "cols"), 64)
    assert e.value.status == U
    assert capi.fsdp_q8_linear_workspace(w, 0) >= 0


def test_null_structs():
    n = ctypes.c_int64()
    lib, none = capi.lib, None
    assert lib.fsdp_q8_quantize(X, 0, 300, none, none, 0) == capi.FSDP_E_INVAL
    assert lib.fsdp_q8_dequantize(none, OUT, 0, 300, 0) == capi.FSDP_E_INVAL
    assert lib.fsdp_q8_product_workspace(none, 0, none, 0, ctypes.byref(n)) == capi.FSDP_E_INVAL
    w = mat(400, 300, "tiles")
    assert lib.fsdp_q8_product_workspace(mat(1, 300), 0, w, 1, none) == capi.FSDP_E_INVAL
    assert lib.fsdp_q8_linear_workspace(none, 1, ctypes.byref(n)) == capi.FSDP_E_INVAL
    assert lib.fsdp_q8_linear_workspace(w, 1, none) == capi.FSDP_E_INVAL
    assert lib.fsdp_q8_linear_backward(w, none, X, 0, 400, 0, OUT, 300, 0, 0, 0, 0, 0) == capi.FSDP_E_INVAL
    assert lib.fsdp_plan_block_scales(none, 0, ctypes.byref(n), ctypes.byref(n)) == capi.FSDP_E_INVAL


def test_copy_in_refusals():
    plan = capi.fsdp_plan_create([s[0] for s in SHAPES], [s[1] for s in SHAPES], 3, 1)
    lib = capi.lib
    assert lib.fsdp_block_scales_shard(None, BASE, 0) == capi.FSDP_E_INVAL
    assert lib.fsdp_pack_allgather_fp8_blocks(None, BASE, BASE, 0) == capi.FSDP_E_INVAL
    assert lib.fsdp_block_scales_shard(plan, BASE, 0) == capi.FSDP_E_STATE
    assert lib.fsdp_pack_allgather_fp8_blocks(plan, BASE, X, 0) == capi.FSDP_E_STATE
    capi.fsdp_plan_destroy(plan)


# ---- the Python checks that need no GPU ---------------------------------------------

def test_q8_names_are_checked():
    t = torch.zeros(4, 8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="blocks"):
        q8.Q8(t, t, "columns")
    with pytest.raises(ValueError, match="format"):
        q8.Q8(t, t, "rows", "e3m4")
    with pytest.raises(ValueError, match="blocks"):
        q8.Q8.empty((4, 8), "tensor", device="cpu")
    q = q8.Q8.empty((130, 33), "rows", device="cpu")
    assert q.shape == (130, 33) and q.codes.shape == (130, 33) and q.codes.stride() == (48, 1)
    assert q.scales_view().shape == (1, 130) and q.c.pitch == 144 and q.nbytes() == 130 * 33 + 130
    assert q8.Q8.empty((0, 5), "cols", device="cpu").scales_view().shape == (0, 0)
