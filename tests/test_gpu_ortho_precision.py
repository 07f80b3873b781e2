"""Precision of the orthogonalisation above 128 rows, for operands of one fp16 part
and of two, on matrices whose roundings are independent and on ones whose
roundings add up.

Tolerance.  Let x be the result before its rounding to bf16, w the exact iterate
and |x - w| <= e |w| in the Frobenius norm.  bf16(x) is the nearest value to x, so no
element of it is further from x than bf16(w)'s is, and |bf16(x) - w| <= |bf16(w) -
w| + 2 |x - w|: the first term is known from w, the second is at most 2 e |w|.

Two parts.  An operand is right to half a step of 22 bits, 2^-22 at most.  X is
rounded to them in each step, and the smallest directions of what that adds are
magnified with X, 485 = 3.4445^5 times at most: 2^-22 485 / 2 = 6e-5.  The
recursion of step_bound, with 2^-22 in the place of 2^-11, gives 4e-5 at the worst
starting value.  Sums in fp32 of at most 3 x 1250 products of 32 elements add
2^-24 for the square root of their number: 4e-6, a few times over.  e = 2^-12.

One part, roundings that add up.  On a matrix of equal singular values s whose
entries all round alike, a step a s + b s^3 + c s^5 with A = s^2 gets from the
rounding of X twice and of A once, half a step u = 2^-11 each, at most 3 u (b s^2 +
2 c s^4) s, and from those of B and X in the product 2 u (b s^2 + c s^4) s; what
came before is multiplied by the step's slope, or across the directions by f(s) / s.

One part, independent roundings.  Half a step over a binade is 0.41 u in the mean
square; the same terms added in squares are at most 1.7 u a step, slopes of about
one carry them on, and five steps are at most 4 u.  The rounding to bf16 is
independent of them: squares add.
"""
import math

import numpy as np
import pytest
import torch

from oracle import muon as M

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("sharded_shard_amd.capi")
from sharded_shard_amd.group import NS_COEFFS, Orthogonalizer  # noqa: E402

DEV = "cuda"
U = 2.0 ** -11
FINE = 2.0 ** -12


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def matrix(shape, seed, kind, dtype):
    g = torch.Generator().manual_seed(seed)
    r, c = shape
    rand = lambda *a: torch.randn(*a, generator=g, dtype=torch.float64)
    if kind == "noise":
        x = rand(r, c)
    elif kind == "falling":
        k = max(1, min(r, c) // 8)
        x = rand(r, k) / torch.arange(1, k + 1) @ rand(k, c) + 0.05 * rand(r, c)
    elif kind == "low":
        x = rand(r, 2) @ rand(2, c)
    elif kind == "constant":
        x = torch.full((r, c), 1.37, dtype=torch.float64)
    elif kind == "signs":                # of rank one
        x = torch.sign(rand(r, 1)) * torch.sign(rand(1, c))
    elif kind == "repeated":             # rows of a wide one, columns of a tall one
        x = rand(1, c).repeat(r, 1) if r <= c else rand(r, 1).repeat(1, c)
    elif kind == "orthonormal":
        q = torch.linalg.qr(rand(max(r, c), min(r, c)))[0]
        x = q if r >= c else q.T
    elif kind == "few":                  # rows that are not zero
        x = torch.zeros(r, c, dtype=torch.float64)
        x[:7] = rand(7, c)
    elif kind == "sparse":
        x = rand(r, c) * (torch.rand(r, c, generator=g, dtype=torch.float64) < 0.01)
    elif kind == "identity":
        x = torch.eye(r, c, dtype=torch.float64)
    else:                                # two constants in blocks
        assert kind == "blocks"
        x = torch.zeros(r, c, dtype=torch.float64)
        x[:r // 2, :c // 2] = 1.0
        x[r // 2:, c // 2:] = -0.61
    return (1e-3 * x).to(dtype).contiguous()


def run(mats, products, coeffs=NS_COEFFS, count=1):
    ins = [m.to(DEV) for m in mats] * count
    outs = [torch.full(m.shape, 7.0, dtype=torch.bfloat16, device=DEV) for m in ins]
    with Orthogonalizer([m.shape for m in ins], coeffs, products=products) as o:
        o.bind(ins, outs)
        o.allocate(torch.full((max(1, o.workspace_bytes),), 0xFF, dtype=torch.uint8, device=DEV))
        o.execute()
        torch.cuda.synchronize()
    return outs


def errors(got, u, coeffs=NS_COEFFS):
    """|got - want|, |bf16(want) - want|, |want|"""
    want = M.orthogonalize(u.double().numpy(), coeffs, 1e-7)
    got = got.cpu().double().numpy()
    assert np.isfinite(got).all()
    near = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    return np.linalg.norm(got - want), np.linalg.norm(near - want), np.linalg.norm(want)


def step_bound(s, coeffs=NS_COEFFS, u=U):
    """Relative error of roundings that all add up, from singular values s."""
    e = 0.0
    for a, b, c in coeffs:
        b, c = b * s * s, c * s ** 4
        slope = max(abs(a + 3 * b + 5 * c), abs(a + b + c))
        e = slope * e + u * s * (3 * abs(b + 2 * c) + 2 * abs(b + c))
        s *= abs(a + b + c)
    return e / s


KINDS = ["noise", "falling", "low", "constant", "signs", "repeated", "orthonormal", "identity", "blocks"]
SHAPES = [(139, 140), (257, 260), (260, 257), (353, 356), (200, 333), (1024, 512), (150, 5000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS + ["few", "sparse"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_two_parts_are_right_on_every_matrix(shape, kind, dtype):
    u = matrix(shape, sum(shape), kind, dtype)
    err, rounding, norm = errors(run([u], "fp16x2")[0], u)
    print("%s %s fp16x2 %.2e of which bf16 %.2e" % (shape, kind, err / norm, rounding / norm))
    assert err <= rounding + 2 * FINE * norm


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS[3:])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_one_part_where_roundings_add_up(shape, kind, dtype):
    u = matrix(shape, sum(shape), kind, dtype)
    s = np.linalg.svd(u.double().numpy(), compute_uv=False)
    s = s[s > 1e-3 * s[0]] / math.sqrt((s * s).sum())
    e = max(step_bound(x) for x in (s[0], s[-1]))
    err, rounding, norm = errors(run([u], "fp16")[0], u)
    print("%s %s fp16 %.2e of which bf16 %.2e, e %.2e" % (shape, kind, err / norm, rounding / norm, e))
    assert err <= rounding + 2 * e * norm


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["noise", "falling"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_one_part_where_roundings_are_independent(shape, kind, dtype):
    """Without X's low part a falling spectrum is 3.5e-3 off before its rounding."""
    u = matrix(shape, sum(shape), kind, dtype)
    err, rounding, norm = errors(run([u], "fp16")[0], u)
    print("%s %s fp16 %.2e of which bf16 %.2e" % (shape, kind, err / norm, rounding / norm))
    assert err <= math.hypot(rounding, 4 * U * norm)


# counts at which a plan takes other tiles for its products
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape,count", [((139, 140), 60), ((1040, 1037), 12), ((677, 680), 40),
                                         ((257, 260), 60), ((440, 523), 40), ((797, 800), 16),
                                         ((900, 7900), 2)], ids=str)
def test_two_parts_in_every_tile_with_edges(shape, count, dtype):
    r, c = shape
    us = [matrix(shape, 11, "falling", dtype), matrix((c, r), 12, "blocks", dtype)]
    outs = run(us, "fp16x2", count=count // 2)
    for u, x in zip(us, outs):
        err, rounding, norm = errors(x, u)
        assert err <= rounding + 2 * FINE * norm, u.shape
    for i, x in enumerate(outs):
        assert torch.equal(x, outs[i % 2]), i


@pytest.mark.parametrize("coeffs", [((1.5, -0.5, 0.0),) * 3, ((2.0, -1.5, 0.5),),
                                    ((8.205, -22.90, 16.46), (4.066, -2.861, 0.518)),
                                    ((1.0, 0.0, 0.0),)], ids=range(4))
@pytest.mark.parametrize("shape", [(260, 180), (30, 50)], ids=lambda s: "%dx%d" % s)
def test_two_parts_with_other_coefficients(coeffs, shape):
    """From singular values of up to 1/8 (noise) no step's slope exceeds its a, and
    what the roundings of 2^-22 add is at most their product 33 times as much."""
    u = matrix(shape, 4, "noise", torch.float32)
    err, rounding, norm = errors(run([u], "fp16x2", coeffs)[0], u, coeffs)
    assert err <= rounding + 2 * FINE * norm


def test_two_parts_over_long_sums():
    for shape in ((130, 40000), (40000, 130)):
        u = matrix(shape, 5, "noise", torch.bfloat16)
        err, rounding, norm = errors(run([u], "fp16x2")[0], u)
        assert err <= rounding + 2 * FINE * norm, shape


@pytest.mark.parametrize("shape", [(150, 200), (200, 150)], ids=lambda s: "%dx%d" % s)
def test_two_parts_on_special_matrices(shape):
    """Zeros stay zeros, what is not finite stays in its matrix, and norms of any
    size lose nothing."""
    z = torch.zeros(shape, dtype=torch.bfloat16)
    u = matrix(shape, 2, "falling", torch.bfloat16)
    bad = [u.clone() for _ in range(3)]
    bad[0][shape[0] // 2, 1] = float("nan")
    bad[1][0, shape[1] - 1] = float("inf")
    bad[2][shape[0] - 1, 0] = float("-inf")
    big = (u.double() * 2.0 ** 120).to(torch.bfloat16)
    outs = run([z, bad[0], u, bad[1], big, bad[2]], "fp16x2")
    assert (outs[0] == 0).all()
    for k in (1, 3, 5):
        assert torch.isnan(outs[k]).all()
    for k, v in ((2, u), (4, big)):
        err, rounding, norm = errors(outs[k], v)
        assert err <= rounding + 2 * FINE * norm


def test_two_parts_in_place_and_captured():
    """In place, and replayed from a graph between eager executions, with the same
    bits."""
    shapes = [(150, 260), (20, 30), (700, 150)]
    mats = [matrix(s, i, "falling", torch.bfloat16) for i, s in enumerate(shapes)]
    want = run(mats, "fp16x2")
    buf = [m.to(DEV) for m in mats]
    ins = [m.to(DEV) for m in mats]
    outs = [torch.empty_like(m) for m in ins]
    with Orthogonalizer(shapes, products="fp16x2") as a, Orthogonalizer(shapes, products="fp16x2") as b:
        a.bind(buf)
        a.execute()
        b.bind(ins, outs)
        b.allocate()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.execute(stream=side)
        for _ in range(3):
            for x in outs:
                x.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            for x, y, w in zip(buf, outs, want):
                assert torch.equal(x, w) and torch.equal(y, w)
            b.execute()
            torch.cuda.synchronize()
        del graph


@pytest.mark.parametrize("kind", ["noise", "falling", "blocks", "signs"])
@pytest.mark.parametrize("shape", [(20, 30), (20, 2000), (2000, 31), (50, 400), (33, 1000), (1000, 64),
                                   (128, 128), (97, 100), (100, 2000), (2000, 128), (70, 20000)],
                         ids=lambda s: "%dx%d" % s)
def test_fp32_inputs_of_few_rows(shape, kind):
    """One slab and several of each of the three classes: 32, 64 and 128 rows."""
    u = matrix(shape, sum(shape), kind, torch.float32)
    err, rounding, norm = errors(run([u], "fp16")[0], u)
    assert err <= rounding + 2 * FINE * norm


# plans whose X X^T is split into parts in tiles of 256 and of 192
@pytest.mark.parametrize("shape,count,products", [((1178, 6738), 5, "fp16"), ((1052, 5818), 6, "fp16"),
                                                  ((2087, 1933), 2, "fp16x2"), ((1035, 1905), 6, "fp16x2")],
                         ids=str)
def test_split_sums_in_the_larger_tiles(shape, count, products):
    r, c = shape
    us = [matrix(shape, 13, "falling", torch.bfloat16), matrix((c, r), 14, "noise", torch.bfloat16)]
    outs = run([us[i % 2] for i in range(count)], products)
    for u, x in zip(us, outs):
        err, rounding, norm = errors(x, u)
        if products == "fp16":
            assert err <= math.hypot(rounding, 4 * U * norm), u.shape
        else:
            assert err <= rounding + 2 * FINE * norm, u.shape
    for i, x in enumerate(outs):
        assert torch.equal(x, outs[i % 2]), i
