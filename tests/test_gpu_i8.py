"""Products of 8-bit integers (mx_i8_quantize, mx_i8_mm) against whole numbers in 64 bits."""
import numpy as np
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}  # half a step, relative


def _codes(x):
    """Codes and scales of fp32 rows, by the definition: fp32 quotients to the nearest even integer."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        s = np.abs(x).max(1) / np.float32(127)
        s = np.where(np.isfinite(x).all(1), s, np.float32(np.nan))
        q = np.where(s[:, None] > 0, np.clip(np.rint(x / s[:, None]), -127, 127), 0)
    return q.astype(np.int8), s.astype(np.float32)


def _weights(torch, N, K, g):
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    return w, torch.exp(torch.randn(N, generator=g, device="cuda")) * 0.01


def _check(torch, y, q, sx, w, sw, tensor_cores):
    """Sums of whole numbers; then two scales, each product and the sum's conversion rounded to fp32, and the result once."""
    q, w = q.double(), w.double()
    total = q @ w.T
    want = total * sx.double()[:, None] * sw.double()
    off = want.abs() * (3 * 2.0 ** -24 + HALF[str(y.dtype)[6:]])
    if tensor_cores:
        # fp32 sums: exact below 2^24; above, each step of 16 products loses at most one place (2^-23) of the sum so far
        most = q.abs() @ w.abs().T
        off = off + torch.where(most < 2.0 ** 24, 0.0, most * (q.shape[1] / 16) * 2.0 ** -23) * sx.double()[:, None] * sw.double()
    err = (y.double() - want).abs()
    assert (err <= off).all(), float((err / off.clamp(min=1e-300)).max())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (2, 8192), (5, 1040), (4, 20000), (130, 512)])
def test_quantize(dtype, M, K):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(K)
    x = (torch.randn((M, K), generator=g, device="cuda") * torch.exp(4 * torch.randn((M, 1), generator=g, device="cuda")))
    x[:, ::7] *= 0.25
    x = x.to(getattr(torch, dtype))
    q, s = ops.i8_quantize(x)
    wq, ws = _codes(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)


def test_quantize_next_to_halves():
    """Values a place or two from half-way between codes."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    rng = np.random.default_rng(3)
    x = np.zeros((40, 4096), np.float32)
    for row in x:
        top = np.float32(np.exp(rng.uniform(-80, 80)))
        s = np.float32(top / np.float32(127))
        row[:] = (rng.integers(-127, 127, 4096) + 0.5).astype(np.float32) * s
        for _ in range(2):
            up = rng.integers(-1, 2, 4096)
            row[:] = np.where(up > 0, np.nextafter(row, np.float32(np.inf)), np.where(up < 0, np.nextafter(row, np.float32(-np.inf)), row))
        row[7] = top
    q, s = ops.i8_quantize(torch.from_numpy(x).cuda())
    wq, ws = _codes(x)
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)


def test_quantize_edges():
    """Zeros, values whose scale is subnormal or vanishes, the largest, halves (to even), NaN and infinities."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    x = torch.zeros((10, 32))
    x[1, 3] = 2.0 ** -149
    x[2, :] = torch.arange(32) * 2.0 ** -147
    x[3, 0], x[3, 1] = torch.finfo(torch.float32).max, -torch.finfo(torch.float32).max
    x[4] = torch.arange(32) / 2 - 8
    x[4, 0] = 127.0
    x[5, 4] = float("nan")
    x[6, 31] = float("inf")
    x[7, 0] = -float("inf")
    x[8] = -0.0
    x[9, 5] = -3.0
    for t in (x, x.bfloat16()):
        q, s = ops.i8_quantize(t.cuda())
        wq, ws = _codes(t.float().numpy())
        assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True) and np.array_equal(q.cpu().numpy(), wq)
    w, sw = _weights(torch, 20, 32, torch.Generator(device="cuda").manual_seed(0))
    for m in (10, 2):  # both kernels' rows: a NaN scale makes its own row NaN
        t = torch.cat([x, x])[-m - 5:][:m] if m == 2 else torch.cat([x, x])
        y = ops.i8_mm(t.cuda(), w, sw, out_dtype=torch.float32)
        bad = ~torch.isfinite(t).all(1)
        assert torch.equal(y.isnan().all(1).cpu(), bad) and torch.equal(y.isnan().any(1).cpu(), bad)


@pytest.mark.parametrize("ydt", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 17, 32), (2, 40, 48), (8, 100, 80), (9, 33, 1040), (16, 250, 8192),
                                   (1, 5000, 64), (3, 2500, 272), (7, 3001, 4096), (1, 10240, 8192), (4, 64, 25600),
                                   (5, 19, 131056), (8, 640, 28672), (3, 330, 40000), (12, 2440, 16384), (17, 5001, 2064),
                                   (24, 999, 8192), (24, 70, 1008), (23, 20, 70000),
                                   (8, 5003, 28672), (13, 200, 28672), (16, 2500, 28672), (6, 33, 40016), (7, 1300, 40016),
                                   (4, 17, 100016), (14, 3000, 14336)])
def test_few_tokens(M, N, K, ydt):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(N + K)
    w, sw = _weights(torch, N, K, g)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    q, sx = ops.i8_quantize(x)
    y = ops.i8_mm(q, w, sw, sx, out_dtype=getattr(torch, ydt))
    _check(torch, y, q, sx, w, sw, M > 8)
    assert torch.equal(y, ops.i8_mm(x, w, sw, out_dtype=getattr(torch, ydt)))
    # the largest codes on both sides
    q = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w[: N // 2] = -128
    w[N // 2:] = 127
    y = ops.i8_mm(q, w, sw, sx, out_dtype=getattr(torch, ydt))
    _check(torch, y, q, sx, w, sw, M > 8)
    assert ops.device_error() == 0


@pytest.mark.parametrize("ydt", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,N,K", [(17, 1, 16), (33, 70, 48), (64, 129, 1040), (70, 300, 8192), (41, 5000, 512), (200, 30000, 64), (100, 1000, 512), (257, 300, 96), (513, 777, 1008),
                                   (600, 512, 4096), (1030, 2500, 80), (4096, 264, 8192), (31, 20, 131056)])
def test_many_tokens(M, N, K, ydt):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(N + K)
    w, sw = _weights(torch, N, K, g)
    x = torch.randn((M, K), generator=g, device="cuda")
    q, sx = ops.i8_quantize(x)
    out = torch.full((M, N), float("nan"), dtype=getattr(torch, ydt), device="cuda")
    y = ops.i8_mm(q, w, sw, sx, out=out)
    assert y is out
    _check(torch, y, q, sx, w, sw, True)
    assert torch.equal(y, ops.i8_mm(x, w, sw, out_dtype=getattr(torch, ydt)))
    q = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    _check(torch, ops.i8_mm(q, w, sw, sx, out_dtype=getattr(torch, ydt)), q, sx, w, sw, True)
    assert ops.device_error() == 0


@pytest.mark.parametrize("M", [1, 8, 40])
def test_weights_quantised_by_the_call_before(M):
    """The product reads its weights as soon as it starts, so not before the quantisation that wrote them has ended."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    N, K = 9000, 4096
    g = torch.Generator(device="cuda").manual_seed(M)
    sources = [torch.randn((N, K), generator=g, device="cuda") for _ in range(4)]
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    xq, sx = ops.i8_quantize(x)
    q, sw = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.zeros(N, device="cuda")
    ys = [[torch.empty((M, N), device="cuda") for _ in range(2)] for _ in sources]
    torch.cuda.synchronize()
    for w, (a, b) in zip(sources, ys):
        ops.i8_quantize(w, q, sw)
        ops.i8_mm(xq, q, sw, sx, out=a)
        ops.i8_quantize(w.neg_(), q, sw)
        ops.i8_mm(x, q, sw, out=b)
    for w, (a, b) in zip(sources, ys):
        wq, sw = ops.i8_quantize(w)
        _check(torch, b, xq, sx, wq, sw, True)
        _check(torch, a, xq, sx, -wq, sw, True)
    assert ops.device_error() == 0


def test_offsets_past_32_bits():
    """Weights of more than 4 GB: their last rows."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    N, K = 600_000, 8192
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    w[-40:] = torch.randint(-128, 128, (40, K), device="cuda", dtype=torch.int8)
    sw = torch.ones(N, device="cuda")
    for M in (1, 20, 300):
        q = torch.randint(-128, 128, (M, K), device="cuda", dtype=torch.int8)
        sx = torch.ones(M, device="cuda")
        y = ops.i8_mm(q, w, sw, sx, out_dtype=torch.float32)
        _check(torch, y[:, -40:], q, sx, w[-40:], sw[-40:], M > 8)
        assert (y[:, :-40] == 0).all()


def test_graphs_streams_and_workspaces():
    """The same bits on every call, in a graph whose tokens change, on two streams at once, in a caller's workspace."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(1)
    N, K = 3000, 2048
    w, sw = _weights(torch, N, K, g)
    for M in (3, 21, 900):
        xs = [torch.randn((M, K), generator=g, device="cuda").bfloat16() for _ in range(3)]
        want = [ops.i8_mm(x, w, sw).clone() for x in xs]
        ws = ops.i8_mm_workspace(M, K)
        ws.fill_(255)
        assert torch.equal(ops.i8_mm(xs[0], w, sw, workspace=ws), want[0])
        x = xs[0].clone()
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            ops.i8_mm(x, w, sw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            y = ops.i8_mm(x, w, sw)
        for i in (1, 2, 0):
            x.copy_(xs[i])
            graph.replay()
            assert torch.equal(y, want[i])
        sts, outs = [torch.cuda.Stream() for _ in range(2)], []
        torch.cuda.synchronize()
        for _ in range(8):
            for i, s in enumerate(sts):
                with torch.cuda.stream(s):
                    outs.append((i, ops.i8_mm(xs[i], w, sw)))
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[i]) for i, o in outs)


def test_a_wait_that_runs_out():
    """The GEMM's bounded waits: NaN and the device error word, then right again."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(2)
    w, sw = _weights(torch, 300, 512, g)
    x = torch.randn((1000, 512), generator=g, device="cuda").bfloat16()  # (so many go to the GEMM)
    want = ops.i8_mm(x, w, sw)
    ops.debug_qmm_stall(True, 20_000_000)
    try:
        y = ops.i8_mm(x, w, sw)
        assert ops.device_error() == 2 and y.isnan().all()
    finally:
        ops.debug_qmm_stall(False)
    assert torch.equal(ops.i8_mm(x, w, sw), want) and ops.device_error() == 0
