"""8-bit matrices as Python holds them: what a view is taken for (no GPU needed)."""
import pytest
import torch

pytest.importorskip("sharded_shard_amd.capi")
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
