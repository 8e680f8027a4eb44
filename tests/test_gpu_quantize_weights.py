"""Weights quantised on the device by the call before the product that reads them: products read their weights as soon as they
start, so not before the quantisation has ended."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("product", ["qmv", "qmv_noalloc", "qmm", "qmm_qx", "moe_qmv", "moe_gate_up_swiglu"])
def test_weights_quantised_by_the_call_before(product, fmt):
    """Several matrices through the same buffers, without a synchronisation, against the same codes made before."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    E, N, K, M = (4 if product.startswith("moe") else 1), 4096, 2048, (40 if product.startswith("qmm") else 2)
    g = torch.Generator(device="cuda").manual_seed(fmt)
    w = torch.randn((E * N, K), generator=g, device="cuda").bfloat16()
    sources = [w, w.neg(), w.flip(1), w.flip(1).neg()]  # (one largest magnitude: NVFP4 tensor scales are alike)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    xq = ops.quantize(fmt, x)
    ids = torch.tensor([[0, 3], [2, 1]], dtype=torch.int32, device="cuda")

    def run(codes, scales):
        if product in ("qmv", "qmv_noalloc", "qmm"):
            return getattr(ops, product)(fmt, codes, scales, x, N)
        if product == "qmm_qx":
            return ops.qmm_qx(fmt, codes, scales, *xq, M, N, K)
        if product == "moe_qmv":
            return ops.moe_qmv(fmt, codes, scales, x, ids, E, N)
        return ops.moe_gate_up_swiglu(fmt, codes, scales, x, ids, E, N // 2)

    # the scales, and of NVFP4 stacks a tensor scale for each expert, of which mx_quantize writes the first
    codes, scales = ops.quantize(fmt, w)
    room = torch.cat([scales, scales[-4:].repeat(E - 1)]) if fmt == 2 else scales.clone()
    want = []
    for s in sources:
        c, q = ops.quantize(fmt, s)
        torch.cuda.synchronize()
        want.append(run(c, torch.cat([q, room[q.numel():]])))
    assert not torch.equal(want[0], want[2])
    torch.cuda.synchronize()
    ys = []
    for s in sources:
        ops.quantize(fmt, s, codes, room[:scales.numel()])
        ys.append(run(codes, room))
    assert all(torch.equal(y, z) for y, z in zip(ys, want))
    assert ops.device_error() == 0
