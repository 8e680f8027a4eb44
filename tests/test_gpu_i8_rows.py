"""8-bit quantisation of more rows than SMs, rows longer than a block's registers hold: both numbers of threads, both types."""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_i8 import _codes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,K", [(152, 2048), (152, 2064), (153, 8192), (153, 8208), (400, 16400), (200, 28672), (170, 32768),
                                 (170, 32784), (160, 65536), (160, 65552)])
def test_many_long_rows(dtype, M, K):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((M, K), generator=g, device="cuda") * torch.exp(4 * torch.randn((M, 1), generator=g, device="cuda"))
    x[5::11, K - 1] *= 100  # (the largest in the last place)
    x[3, K - 2], x[4, 0], x[6] = float("nan"), float("inf"), 0.0
    x = x.to(getattr(torch, dtype))
    q, s = ops.i8_quantize(x)
    wq, ws = _codes(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True) and np.array_equal(q.cpu().numpy(), wq)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,N,K", [(300, 200, 16400), (200, 3000, 28672)])
def test_products_of_many_long_rows(dtype, M, N, K):
    """The quantisation on the way (to f16 integers) as before the call."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((M, K), generator=g, device="cuda").to(getattr(torch, dtype))
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.ones(N, device="cuda")
    q, sx = ops.i8_quantize(x)
    y = ops.i8_mm(x, w, sw, out_dtype=torch.float32)
    assert torch.equal(y, ops.i8_mm(q, w, sw, sx, out_dtype=torch.float32))
    want = (q.double() @ w.double().T).float() * sx[:, None]  # (sums of a few 10^5: exact in fp32)
    assert torch.equal(y, want) and ops.device_error() == 0
