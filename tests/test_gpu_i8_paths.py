"""Products of 8-bit integers, way by way: which kernels a size takes, as the graph of a captured call names them, and that the
result is the exact sum of whole numbers, rounded to fp32, times one scale and then the other, rounded after each."""
import re

import pytest

from gpu_util import need_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:DEBUG")]

# streaming passes by single CTAs or pairs (groups of 8 tokens), and the GEMM's tiles
KINDS = {r"i8_mv_kernelILi1E\wLb0E": "stream 8", r"i8_mv_kernelILi2E\wLb0E": "stream 16", r"i8_mv_kernelILi1E\wLb1E": "pairs 8",
         r"i8_mv_kernelILi2E\wLb1E": "pairs 16", r"qmm_kernelILi3ELi1ELi3E": "few rows", r"qmm_kernelILi3ELi1ELi0E": "tiles of 256",
         r"qmm_kernelILi3ELi2ELi0E": "tiles of 512"}


def _ways(torch, call, tmp_path):
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph, stream=st):
        call()
    graph.debug_dump(str(tmp_path / "graph.dot"))
    names = re.findall(r"_ZN2mx\w+", (tmp_path / "graph.dot").read_text())
    return [kind for n in names for pattern, kind in KINDS.items() if re.search(pattern, n)]


def _exact(torch, y, q, sx, w, sw, sums_in_fp32):
    total = q.double() @ w.double().T
    if sums_in_fp32:  # exact while every partial sum stays below 2^24: after each 64 of K, and 64 products more
        M, K = q.shape
        blocks = -(-K // 64)
        pad = lambda t: torch.nn.functional.pad(t.double(), (0, 64 * blocks - K)).view(t.shape[0], blocks, 64).transpose(0, 1)  # noqa: E731
        partial = torch.bmm(pad(q), pad(w).transpose(1, 2)).cumsum(0).abs().max()
        assert float(partial) + 64 * 128 * 128 < 2.0 ** 24
    want = (total.float() * sx[:, None]) * sw
    assert torch.equal(y, want.to(y.dtype))


SIZES = [(1, 2500, 4096), (5, 17, 48), (8, 999, 8192), (3, 330, 40000), (9, 2500, 4096), (13, 33, 1040), (16, 2440, 8192),
         (24, 999, 8192), (8, 5003, 28672), (7, 1300, 40016), (13, 2500, 28672), (16, 2500, 28672), (64, 5000, 1024),
         (128, 10001, 2064), (33, 20000, 512), (100, 3000, 40000), (300, 700, 1008), (129, 1000, 4096), (1030, 20000, 80)]


def _operands(torch, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    return torch.randn((M, K), generator=g, device="cuda").bfloat16(), w, torch.exp(torch.randn(N, generator=g, device="cuda")) * 0.01


def test_every_way_is_taken(tmp_path):
    """An estimate that changes leaves no kernel without a size here."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    taken = {}
    for M, N, K in SIZES:
        x, w, sw = _operands(torch, M, N, K)
        ways = _ways(torch, lambda: ops.i8_mm(x, w, sw), tmp_path)
        assert ways, (M, N, K)
        taken.update({way: (M, N, K) for way in ways})
    assert set(taken) == set(KINDS.values())


@pytest.mark.parametrize("ydt", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_exact_sums(M, N, K, ydt, tmp_path):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    ydt = getattr(torch, ydt)
    x, w, sw = _operands(torch, M, N, K)
    q, sx = ops.i8_quantize(x)
    ways = _ways(torch, lambda: ops.i8_mm(q, w, sw, sx), tmp_path)
    assert _ways(torch, lambda: ops.i8_mm(x, w, sw), tmp_path) == ways
    whole_numbers = all(way.startswith(("stream", "pairs")) for way in ways)
    got = ops.i8_mm(q, w, sw, sx, out_dtype=ydt)
    _exact(torch, got, q, sx, w, sw, not whole_numbers)
    assert torch.equal(got, ops.i8_mm(x, w, sw, out_dtype=ydt))
    if whole_numbers:  # sums up to 2^14 K, far past 2^24
        q.fill_(-128)
        w[::2] = -128
        w[1::2, : K // 2 + 3] = 127
        _exact(torch, ops.i8_mm(q, w, sw, sx, out_dtype=ydt), q, sx, w, sw, False)
    assert ops.device_error() == 0


@pytest.mark.parametrize("M,N,K", [(64, 5000, 1024), (33, 20000, 512), (128, 10001, 2064)])
def test_a_wait_that_runs_out_in_a_tile_of_few_rows(M, N, K):
    """NaN in every row and column, the device error word, then right again."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    x, w, sw = _operands(torch, M, N, K)
    want = ops.i8_mm(x, w, sw)
    for dtype in (torch.bfloat16, torch.float32):
        ops.debug_qmm_stall(True, 20_000_000)
        try:
            y = ops.i8_mm(x, w, sw, out_dtype=dtype)
            assert ops.device_error() == 2 and y.isnan().all()
        finally:
            ops.debug_qmm_stall(False)
    assert torch.equal(ops.i8_mm(x, w, sw), want) and ops.device_error() == 0
