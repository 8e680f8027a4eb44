"""The beams' selection where a row's logits rise with the token: more vectors reach a step's bound than the queue and the
list hold, so pieces go the exact way."""
import numpy as np
import pytest

import serve_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

OFF = 2.0 ** -16  # a key's distance beside its rounding, as derived in test_gpu_beam.py


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,W,V,k,masked", [(1, 4, 40000, 8, False), (3, 4, 33001, 16, True), (1, 16, 20000, 128, False),
                                            (2, 8, 17003, 128, True), (1, 1, 300000, 100, False)])
def test_rising_rows(dtype, B, W, V, k, masked):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn((B * W, V), generator=g, device="cuda") * 3).sort(1).values
    x[1::3] = x[1::3].flip(1)  # (some fall)
    x = x.to(getattr(torch, dtype))
    c = torch.randn((B, W), generator=g, device="cuda") - 9
    allowed, mask = None, None
    if masked:
        allowed = np.random.default_rng(V).random((B * W, V)) < 0.7
        bits = np.zeros((B * W, -(-V // 32) * 32), np.uint8)
        bits[:, :V] = allowed
        mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32)).cuda()
    got = ops.beam_select(x, c, k, V - 1, mask)
    want = ref.beam_candidates(x.double().cpu().numpy(), c.double().cpu().numpy().reshape(-1), W, allowed)
    ref.check_beams(got, want, W, k, V - 1, OFF)
    again = ops.beam_select(x, c, k, V - 1, mask)
    assert all(torch.equal(a, b) for a, b in zip(got, again)) and ops.device_error() == 0
