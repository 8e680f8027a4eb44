"""Rotary positions where the arguments are unusual: no rotation."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("gap", [0, 3])
def test_no_rotation_is_a_copy(dtype, gap):
    """Without a table no position is wrong, as in the append."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    x = torch.randn((5, 3 * 64 + gap), device="cuda").to(getattr(torch, dtype))[:, :192].unflatten(1, (3, 64))
    pos = torch.tensor([0, 7, -1, 1 << 30, 2], dtype=torch.int32, device="cuda")
    for table in (None, torch.empty((0, 0, 2), device="cuda"), torch.empty((3, 0, 2), device="cuda")):
        assert torch.equal(ops.rope(x, pos, table), x)
    assert ops.device_error() == 0
