"""8-bit matrices as Python holds them: what a view is taken for (no GPU needed)."""
import ctypes

import pytest
import torch

capi = pytest.importorskip("sharded_shard_amd.capi")
from sharded_shard_amd import q8  # noqa: E402


@pytest.mark.parametrize("dtype,named", [(torch.float8_e5m2, "e4m3"), (torch.float8_e4m3fn, "e5m2")])
@pytest.mark.parametrize("blocks", ["tensor", "tiles"])
def test_a_float8_type_is_its_format(dtype, named, blocks):
    """Codes of one float8 type are not read as those of the other, whose values differ."""
    t = torch.zeros(4, 16, dtype=torch.uint8)
    scales = None if blocks == "tensor" else torch.zeros(1, 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="float8.* codes are not " + named):
        q8.Q8(t.view(dtype), scales, blocks, named)
    if named == "e4m3":
        with pytest.raises(ValueError, match="float8.* codes are not e4m3"):
            q8.Q8(t.view(dtype), scales, blocks)


def empty(rows, cols, blocks="tiles", format="e4m3"):
    return q8.Q8.empty((rows, cols), blocks, format, device="cpu")


def odd(rows, cols):
    """A weight whose codes lie at an odd address: products copy it into their workspace."""
    q = empty(rows, cols)
    c = capi.Q8Struct.from_buffer_copy(q.c)
    c.codes, c.ld = c.codes + 1, c.ld + 1
    q.c, q.aligned = c, False
    return q


def test_another_weight_has_its_own_workspace():
    """What a layer keeps about its weight goes when the weight does."""
    layer = q8.Linear8(empty(256, 512))
    ws, n = layer._workspace(64, None)
    assert n == ws.numel() == capi.fsdp_q8_linear_workspace(layer.weight.c, 64)
    for w in (odd(256, 512), empty(1024, 512), empty(256, 512)):
        layer.weight = w
        ws, n = layer._workspace(64, None)
        assert n == ws.numel() == capi.fsdp_q8_linear_workspace(w.c, 64)
    assert layer.weight is w
    # the constructor's checks
    with pytest.raises(ValueError, match="blocks"):
        layer.weight = empty(256, 512, "rows")
    with pytest.raises(ValueError, match="E4M3"):
        layer.weight = empty(256, 512, "tiles", "e5m2")
    assert layer.weight is w


def test_what_a_layer_keeps_does_not_grow_without_end():
    layer = q8.Linear8(empty(1, 16))
    for tokens in range(1, 5000):
        layer._workspace(tokens, None)
    assert len(layer._bytes) <= 4096


def test_how_a_product_is_cut_up():
    """The sizes whose tiles the GPU tests rely on; refusals as the product's."""
    cut = lambda m, n, k, ta, tb: capi.fsdp_q8_product_cut(
        empty(*((k, m) if ta else (m, k)), "cols" if ta else "rows").c, int(ta),
        empty(*((n, k) if tb else (k, n)), "tiles").c, int(tb))
    assert cut(1, 14336, 4096, False, True) == cut(32, 64, 128, False, True) == (0, 1)
    assert cut(32, 28672, 8192, False, True)[0] == 64       # tiles read as many weights faster
    for ta, tb in ((False, True), (False, False), (True, False)):
        assert cut(8192, 4096, 4096, ta, tb) == (256, 1)
        assert cut(3520, 5824, 384, ta, tb) == (256, 1)
        assert cut(64, 64, 256, ta, tb)[0] == 64
        assert cut(256, 256, 8200, ta, tb)[1] > 1
    with pytest.raises(capi.FsdpError):
        capi.fsdp_q8_product_cut(empty(4, 16, "rows").c, 1, empty(4, 16).c, 1)
    lib, n = capi.lib, ctypes.c_int32()
    a, b = empty(4, 16, "rows").c, empty(4, 16).c
    assert lib.fsdp_q8_product_cut(a, 0, b, 1, None, ctypes.byref(n)) == capi.FSDP_E_INVAL
    assert lib.fsdp_q8_product_cut(None, 0, b, 1, ctypes.byref(n), ctypes.byref(n)) == capi.FSDP_E_INVAL
