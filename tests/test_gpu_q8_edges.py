"""8-bit matrices on the GPU, at the edges: signs of zero, single rows far apart,
checkpoints at odd addresses."""
import numpy as np
import pytest
import torch

from oracle import q8 as Q

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("sharded_shard_amd.capi")
from sharded_shard_amd import q8  # noqa: E402
from sharded_shard_amd.group import ShardedGroup  # noqa: E402

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def zeros_of_both_signs(rows, cols):
    """Every third element a zero, of either sign; also values that round to one."""
    g = np.random.default_rng([rows, cols])
    x = g.standard_normal((rows, cols)).astype(np.float32)
    pick = g.integers(0, 6, (rows, cols))
    x[pick == 0], x[pick == 1] = 0.0, -0.0
    x[pick == 2] *= np.float32(2.0 ** -40)
    return x


@pytest.mark.parametrize("shape", [(130, 40), (256, 384), (33, 129)], ids=str)
def test_copy_in_keeps_the_sign_of_zero(shape):
    """The codes themselves, as the quantiser makes them."""
    x = zeros_of_both_signs(*shape)
    g = ShardedGroup([shape], 1, 0)
    g.shard_view(g.master_flat, 0).copy_(torch.from_numpy(x.reshape(-1)))
    scales = torch.empty(g.n_block_scales, dtype=torch.uint8, device=DEV)
    seg = torch.empty(g.S, dtype=torch.uint8, device=DEV)
    g.block_scales(scales)
    g.pack_fp8_blocks(seg, scales)
    codes, _ = Q.quantize(x, "tiles", "e4m3")
    assert np.array_equal(codes & 128, np.signbit(x) * 128)
    assert np.array_equal(seg.cpu().numpy()[:x.size].reshape(shape), codes)
    g.close()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(130, 40), (256, 384), (33, 129)], ids=str)
def test_the_quantiser_keeps_the_sign_of_zero(shape, dtype, fmt):
    x = torch.from_numpy(zeros_of_both_signs(*shape)).to(DEV, dtype)
    h = x.double().cpu().numpy()
    for blocks in ("rows", "cols", "tiles"):
        codes, _ = Q.quantize(h, blocks, fmt)
        assert np.array_equal(codes & 128, np.signbit(h) * 128)
        assert np.array_equal(q8.quantize(x, blocks, fmt).codes_view().cpu().numpy(), codes)
    for q, blocks in zip(q8.quantize(x, "both", fmt), ("rows", "cols")):
        assert np.array_equal(q.codes_view().cpu().numpy(), Q.quantize(h, blocks, fmt)[0])


@pytest.mark.parametrize("stride", [1100 * 4096, 1100 * 4096 + 1])
def test_one_row_however_far_the_next_would_be(stride):
    """The last token of a long sequence, [1, tokens, width][:, -1]: its stride is the sequence's."""
    g = torch.Generator(device=DEV).manual_seed(1)
    flat = torch.randn(stride + 4096, generator=g, device=DEV).bfloat16()
    row = flat.as_strided((1, 4096), (stride, 1), 8)
    same = row.clone()
    w = q8.quantize(torch.randn(300, 4096, generator=g, device=DEV).bfloat16(), "tiles")
    for blocks in ("rows", "cols", "tiles"):
        a, b = q8.quantize(row, blocks), q8.quantize(same, blocks)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        out = torch.zeros_like(flat).as_strided((1, 4096), (stride, 1), 3)
        assert torch.equal(q8.dequantize(a, out=out), q8.dequantize(b))
    codes = torch.zeros(stride + 4096, dtype=torch.uint8, device=DEV).as_strided((1, 4096), (stride, 1), 0)
    a = q8.quantize(same, "rows")
    codes.copy_(a.codes)
    far = q8.Q8(codes, a.scales, "rows")
    want = q8.product(a, w, trans_b=True)
    assert torch.equal(q8.product(far, w, trans_b=True), want)
    assert torch.equal(q8.dequantize(far), q8.dequantize(a))
    out = torch.zeros(stride, dtype=torch.bfloat16, device=DEV).as_strided((1, 300), (stride, 1), 0)
    assert torch.equal(q8.product(a, w, trans_b=True, out=out), want)
    one, two = q8.Linear8(w), q8.Linear8(w)
    assert torch.equal(one.forward(row, out=out), two.forward(same))
    dy = torch.randn(stride, generator=g, device=DEV).bfloat16().as_strided((1, 300), (stride, 1), 0)
    dw = [torch.empty(300, 4096, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    dx = torch.zeros(stride, dtype=torch.bfloat16, device=DEV).as_strided((1, 4096), (stride, 1), 0)
    assert torch.equal(one.backward(dy, dw[0], out=dx), two.backward(dy.clone(), dw[1]))
    assert torch.equal(*dw)


@pytest.mark.parametrize("at,more", [(1, 0), (3, 5), (16, 1), (8, 16)])
@pytest.mark.parametrize("tokens", [40, 333, 1500])
def test_backward_of_a_checkpoint_at_any_address(tokens, at, more):
    """The native step with a caller's own checkpoint, in exactly its workspace: the bits of the
    separate calls on one that lies as Linear8 lays it."""
    n, k = 260, 515
    g = torch.Generator(device=DEV).manual_seed(tokens)
    x, dy = (torch.randn(tokens, c, generator=g, device=DEV).bfloat16() for c in (k, n))
    w = q8.quantize(torch.randn(n, k, generator=g, device=DEV).bfloat16(), "tiles")
    saved = q8.quantize(x, "cols")
    ld = -(-k // 16) * 16 + more
    codes = torch.full((at + tokens * ld,), 0x7F, dtype=torch.uint8, device=DEV)
    codes = codes[at:].view(tokens, ld)[:, :k]
    codes.copy_(saved.codes)
    far = q8.Q8(codes, saved.scales, "cols")
    need = capi.fsdp_q8_linear_workspace(w.c, tokens)
    buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    ws = buf[256:256 + need]
    dx = torch.empty(tokens, k, dtype=torch.bfloat16, device=DEV)
    dw = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    capi.fsdp_q8_linear_backward(w.c, far.c, dy.data_ptr(), capi.FSDP_DTYPE_BF16, n, capi.FSDP_Q8_E4M3,
                                 dx.data_ptr(), k, dw.data_ptr(), k, ws.data_ptr(), need)
    dr, dc = q8.quantize(dy, "both")
    assert torch.equal(dx, q8.product(dr, w))
    assert torch.equal(dw, q8.product(dc, saved, trans_a=True))
    assert (buf[:256] == 0x5A).all() and (buf[256 + need:] == 0x5A).all()


def test_results_beside_their_operands():
    """x, y, dy and dx as columns of one buffer: each written without a byte of the others."""
    t, n, k = 130, 96, 72
    g = torch.Generator(device=DEV).manual_seed(3)
    buf = torch.randn(t, k + n + n + k, generator=g, device=DEV).bfloat16()
    x, y, dy, dx = buf.split((k, n, n, k), 1)
    was = buf.clone()
    w = q8.quantize(torch.randn(n, k, generator=g, device=DEV).bfloat16(), "tiles")
    layer, alone = q8.Linear8(w), q8.Linear8(w)
    dw = [torch.empty(n, k, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    want_y = alone.forward(x.clone())
    want_dx = alone.backward(dy.clone(), dw[1])
    assert torch.equal(layer.forward(x, out=y), want_y)
    assert torch.equal(layer.backward(dy, dw[0], out=dx), want_dx) and torch.equal(*dw)
    assert torch.equal(buf[:, :k], was[:, :k]) and torch.equal(dy, was[:, k + n:k + 2 * n])
    with pytest.raises(capi.FsdpError):
        layer.forward(x, out=buf[:, k - 1:k - 1 + n])
