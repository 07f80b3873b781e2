"""Products of 8-bit matrices in every tile, cut and form: whole numbers bit for bit, what
the matrix instruction keeps of neighbouring products, and the error of the sums before
they are rounded to bf16."""
import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("sharded_shard_amd.capi")
from sharded_shard_amd import q8  # noqa: E402

DEV = "cuda"
FORMS = [(False, True), (False, False), (True, False)]       # x W^T, dy W, dy^T x
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def held(values, exponents, blocks, fmt):
    """A matrix with these numbers as codes and 2^exponents for its blocks; NaN in all memory
    of it that holds neither."""
    rows, cols = values.shape
    q = q8.Q8.empty((rows, cols), blocks, fmt)
    q._both.fill_(0x7F)
    q._both[rows * q.c.ld:].fill_(0xFF)
    q.codes.copy_(values.to(FLOAT8[fmt]).view(torch.uint8))
    q.scales.copy_((exponents + 127).to(torch.uint8))
    return q


def worth(values, exponents, blocks):
    """What they stand for, in fp64."""
    rows, cols = values.shape
    e = exponents.t() if blocks == "rows" else exponents
    if blocks in ("rows", "tiles"):
        e = e.repeat_interleave(128, 1)[:, :cols]
    if blocks in ("cols", "tiles"):
        e = e.repeat_interleave(128, 0)[:rows]
    return values.double() * torch.exp2(e.double())


def whole(rows, cols, blocks, fmt, most, exps, seed):
    """Whole numbers up to `most`, blocks of 2^0 to 2^(exps - 1)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = torch.randint(-most, most + 1, (rows, cols), generator=g, device=DEV, dtype=torch.int8).float()
    e = torch.randint(0, exps, q8.scale_lines(rows, cols, blocks), generator=g, device=DEV)
    return held(v, e, blocks, fmt), worth(v, e, blocks)


def cut(a, b, ta, tb):
    return capi.fsdp_q8_product_cut(a.c, int(ta), b.c, int(tb))


def walks(m, n, k, tile, split):
    """Whether a block takes more than one tile: those that fit the device at once are 256, two
    for 128 and four for 64 times as many, and every stretch has two steps."""
    items = -(-m // tile) * -(-n // tile) * split
    return items > 256 * {256: 1, 128: 2, 64: 4}[tile] and -(-k // 128) // split >= 2


def check_whole(m, n, k, ta, tb, fmt, blocks_b, most, exps, want):
    # every sum of products is a whole number under 2^24: exact in any order
    assert most * most * 4 ** (exps - 1) * k < 1 << 24
    blocks_a = "cols" if ta else "rows"
    a, av = whole(*((k, m) if ta else (m, k)), blocks_a, fmt, most, exps, 1)
    b, bv = whole(*((n, k) if tb else (k, n)), blocks_b, "e4m3", most, exps, 2)
    tile, split = cut(a, b, ta, tb)
    assert (tile, split > 1, tile > 0 and walks(m, n, k, tile, split)) == want, (tile, split)
    got = q8.product(a, b, ta, tb)
    av = av.t().contiguous() if ta else av
    bv = bv.t().contiguous() if tb else bv
    for j in range(0, n, 8192):         # (of the right operand a part at a time)
        exact = av @ bv[:, j:j + 8192].contiguous()
        assert torch.equal(got[:, j:j + 8192], exact.bfloat16()), (m, n, k, ta, tb, fmt, blocks_b, j)


# rows, columns, inner; the tile, whether the sum is cut, whether blocks go from tile to tile
CUTS = [
    ((33, 64, 64), (64, False, False)),
    ((257, 511, 300), (64, False, False)),
    ((128, 128, 2048), (64, True, False)),
    ((100, 130, 2045), (64, True, False)),
    ((40, 70000, 200), (64, False, True)),
    ((70001, 40, 299), (64, False, True)),
    ((2049, 2305, 272), (128, False, False)),
    ((1000, 2049, 100), (128, False, False)),
    ((130, 1500, 8200), (128, True, False)),
    ((8000, 2049, 300), (128, False, True)),
    ((4300, 4500, 400), (128, False, True)),
    ((1000, 8200, 16), (256, False, False)),
    ((1001, 8200, 400), (256, False, False)),
    ((3517, 5821, 200), (256, False, True)),
    ((3520, 5824, 384), (256, False, True)),
    ((3517, 5821, 387), (256, False, True)),
    ((5000, 4500, 1300), (256, False, True)),
    ((8191, 4097, 1153), (256, False, True)),
]


@pytest.mark.parametrize("ta,tb", FORMS, ids=["xWt", "dyW", "dytx"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("mnk,want", CUTS, ids=str)
def test_whole_numbers_are_exact(mnk, want, ta, tb, fmt):
    for blocks_b in ("rows" if tb else "cols", "tiles"):
        check_whole(*mnk, ta, tb, fmt, blocks_b, 4, 4 if mnk[2] <= 8200 else 2, want)


@pytest.mark.parametrize("ta,tb", FORMS, ids=["xWt", "dyW", "dytx"])
@pytest.mark.parametrize("mnk,want", [((40, 70000, 16000), (64, True, True)),
                                      ((200, 4000, 65536), (256, True, False)),
                                      ((200, 20000, 65536), (256, True, True))], ids=str)
def test_long_sums_of_whole_numbers_are_exact(mnk, want, ta, tb):
    check_whole(*mnk, ta, tb, "e4m3", "tiles", 2, 2, want)


@pytest.mark.parametrize("mnk", [(1, 64, 128), (5, 33, 47), (16, 1000, 256), (1, 5000, 4100),
                                 (16, 6001, 900), (32, 129, 1024), (17, 4096, 1299), (32, 6000, 1024),
                                 (20, 8190, 2100)], ids=str)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_few_rows_of_whole_numbers_are_exact(mnk, fmt):
    for blocks_b in ("rows", "tiles"):
        check_whole(*mnk, False, True, fmt, blocks_b, 4, 4, (0, False, False))


# (1 x 28000 is 438 tiles in four stretches, 1752 for the 1024 blocks that fit at once)
@pytest.mark.parametrize("mnk,want", [((32, 256, 8192), (64, True, False)), ((17, 9000, 130), (64, False, False)),
                                      ((20, 8200, 4100), (64, True, False)),
                                      ((1, 28000, 8192), (64, True, True))], ids=str)
def test_few_rows_by_tiles_of_whole_numbers_are_exact(mnk, want):
    """Where tiles are faster: long sums, many columns."""
    check_whole(*mnk, False, True, "e4m3", "tiles", 4, 4, want)


# ---- what the instruction keeps ------------------------------------------------------

def pattern(n, k):
    """[n, k]: in one eight of each line 2^8 and seven times 2^-5, 13 powers of two below; the
    2^8 is taken away again by another eight.  The sum is 7 2^-5, if all 13 are kept."""
    v = torch.zeros(n, k)
    eights = k // 8
    for i in range(n):
        e = i // 8 % eights
        v[i, 8 * e:8 * e + 8] = 2.0 ** -5
        v[i, 8 * e + i % 8] = 2.0 ** 8
        v[i, 8 * ((e + eights // 2) % eights) + 5 * i % 8] = -2.0 ** 8
    return v.to(DEV)


@pytest.mark.parametrize("ta,tb", FORMS, ids=["xWt", "dyW", "dytx"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("mnk,tile", [((20, 64, 1024), 0), ((100, 120, 1024), 64), ((2049, 2305, 272), 128),
                                      ((3517, 5821, 384), 256)], ids=str)
def test_products_13_powers_of_two_below_the_largest_of_eight_are_kept(mnk, tile, ta, tb, fmt):
    m, n, k = mnk
    turn = lambda v, t: v.t().contiguous() if t else v
    zeros = lambda q: torch.zeros(q8.scale_lines(*q[0], q[1]), dtype=torch.int64, device=DEV)
    ba, bb = ("cols" if ta else "rows"), ("rows" if tb else "cols")
    for in_a in (True, False):
        av = pattern(m, k) if in_a else torch.ones(m, k, device=DEV)
        bv = torch.ones(n, k, device=DEV) if in_a else pattern(n, k)
        av, bv = turn(av, ta), turn(bv, not tb)
        a = held(av, zeros((av.shape, ba)), ba, fmt)
        b = held(bv, zeros((bv.shape, bb)), bb, "e4m3")
        if tile or (tb and not ta):
            assert cut(a, b, ta, tb)[0] == tile
        got = q8.product(a, b, ta, tb)
        assert (got.float() == 7 * 2.0 ** -5).all(), (in_a, got.float().unique()[:8])


@pytest.mark.parametrize("ta,tb", FORMS, ids=["xWt", "dyW", "dytx"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("k", [2048, 8192, 65536])
def test_the_error_of_sums_of_normal_data(k, fmt, ta, tb):
    """The fp32 sums of a product that is cut into stretches lie in its workspace.  A product
    loses less than 2^-13 of the power of two of the largest of its eight, p say, seven of an
    eight at most: where the losses' signs are as random as the products', an eight is off
    by sqrt(7) 2^-13 p (root mean square) at most, and p^2 is at most the sum of the eight's
    squares.  Over the eights of independent operands that is sqrt(7) 2^-13 of the results'
    root mean square; and the fp32 additions, as in the oracle's bound, each 2^-24 of sums no
    larger than the results' own, ten standard deviations allowed."""
    m = n = 256
    g = torch.Generator(device=DEV).manual_seed(k)
    of = lambda rows, cols, blocks, f: q8.quantize(
        torch.randn(rows, cols, generator=g, device=DEV).bfloat16(), blocks, f)
    a = of(*((k, m) if ta else (m, k)), "cols" if ta else "rows", fmt)
    b = of(*((n, k) if tb else (k, n)), "rows" if tb else "cols", "e4m3")
    split = cut(a, b, ta, tb)[1]
    assert split > 1
    ws = torch.empty(capi.fsdp_q8_product_workspace(a.c, int(ta), b.c, int(tb)), dtype=torch.uint8, device=DEV)
    assert ws.numel() == 4 * m * n * split
    got = q8.product(a, b, ta, tb, workspace=ws)
    av, bv = (q8.dequantize(q, torch.float32).double() for q in (a, b))
    exact = (av.t() if ta else av).contiguous() @ (bv.t() if tb else bv).contiguous()
    sums = ws.view(torch.float32).view(split, m, n).double().sum(0)
    rms = lambda x: x.pow(2).mean().sqrt().item()
    adds = k / 8 + k / 128 + 24
    assert rms(sums - exact) <= (7 ** 0.5 * 2.0 ** -13 + 10 * adds * 2.0 ** -24) * rms(exact)
    # and the one rounding that is left: 2^-8 of the joined sum, whose additions are fp32
    room = 2.0 ** -8 * sums.abs() + (1 + 2.0 ** -8) * split * 2.0 ** -24 * ws.view(torch.float32).view(
        split, m, n).double().abs().sum(0)
    assert ((got.double() - sums).abs() <= room).all()
