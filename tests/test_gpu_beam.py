"""The beams' selection (mx_beam_select) against 64 bits: sizes, types, strides and alignments, masks, beams without
candidates, ties, ends, streams and graphs."""
import math

import numpy as np
import pytest

import serve_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

# A key's distance from the exact one beside its rounding to fp32.  The logarithm of a sum of exponentials moves by the
# sum's relative error: e^(x - m) with |x - m| < 32 where it counts is off by 2^-22 (the exponential) and by the
# rounding of x - m and of its product with log2 e, 32 (2^-24 + 2^-24); up to 64 additions in a thread, 16 in the block,
# 2^-24 each: below 2^-22 + 2^-18 + 2^-17 < 2^-16.
OFF = 2.0 ** -16


def _run(torch, logits, scores, k=None, eos=-1, allowed=None, mask=None, **kw):
    from gemm_decode_register_gb300 import ops

    B, W = scores.shape
    k = 2 * W if k is None else k
    got = ops.beam_select(logits, scores, k, eos, mask, **kw)
    want = ref.beam_candidates(logits.double().cpu().numpy(), scores.double().cpu().numpy().reshape(-1), W, allowed)
    ref.check_beams(got, want, W, k, eos, OFF)
    assert ops.device_error() == 0
    return got


def _mask(torch, allowed):
    rows, V = allowed.shape
    bits = np.zeros((rows, -(-V // 32) * 32), np.uint8)
    bits[:, :V] = allowed
    words = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
    return torch.from_numpy(np.ascontiguousarray(words)).cuda()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,W,V,k", [
    (1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 2, 7), (1, 4, 31, 8), (3, 2, 257, 128), (2, 5, 1000, 10), (1, 64, 300, 128),
    (5, 4, 4099, 8), (1, 1, 40000, 2), (1, 2, 33000, 128), (40, 3, 17000, 6), (300, 1, 700, 2), (3, 16, 50001, 33)])
def test_sizes(dtype, B, W, V, k):
    torch = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(B * 100 + V)
    x = (torch.randn((B * W, V), generator=g, device="cuda") * 3).to(getattr(torch, dtype))
    c = torch.randn((B, W), generator=g, device="cuda") * 2 - 20
    _run(torch, x, c, k, eos=V // 2)


@pytest.mark.parametrize("dtype,lead,pad", [("bfloat16", 1, 0), ("bfloat16", 3, 6), ("bfloat16", 8, 5), ("float32", 1, 2),
                                            ("float32", 2, 1), ("float32", 0, 3)])
def test_rows_of_any_stride_and_alignment(dtype, lead, pad):
    torch = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    whole = torch.randn((6, 5003 + lead + pad), generator=g, device="cuda").to(getattr(torch, dtype))
    whole[:, :lead] = 1e4  # what lies beside a row must not count
    whole[:, lead + 5003:] = math.inf
    c = torch.zeros((2, 3), device="cuda")
    _run(torch, whole[:, lead:lead + 5003], c)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_masks(dtype):
    """Beams that may take half of the tokens, few, one, the last one, none; what is masked may hold anything."""
    torch = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(4)
    W, V = 6, 20011
    x = (torch.randn((2 * W, V), generator=g, device="cuda") * 3).to(getattr(torch, dtype))
    rng = np.random.default_rng(4)
    allowed = rng.random((2 * W, V)) < np.array([0.5, 0.01, 0.0, 0.0, 0.0, 1.0] * 2)[:, None]
    allowed[2, 7] = allowed[3, V - 1] = allowed[8, 31] = True
    hidden = ~torch.from_numpy(allowed).cuda()
    x[0, hidden[0]] = math.nan
    x[1, hidden[1]] = math.inf
    x[6, hidden[6]] = torch.finfo(x.dtype).max
    x[7, hidden[7]] = torch.finfo(x.dtype).min
    c = torch.randn((2, W), generator=g, device="cuda")
    _run(torch, x, c, 12, 5, allowed, _mask(torch, allowed))
    wide = torch.zeros((2 * W, 800), dtype=torch.int32, device="cuda")  # rows of a wider mask
    m = _mask(torch, allowed)
    wide[:, 5:5 + m.shape[1]] = m
    _run(torch, x[:, :], c, 12, 5, allowed, wide[:, 5:5 + m.shape[1]])


def test_nothing_allowed_anywhere():
    torch = need_gpu()
    x = torch.zeros((4, 100), device="cuda")
    allowed = np.zeros((4, 100), bool)
    got = _run(torch, x, torch.zeros((2, 2), device="cuda"), 3, 0, allowed, _mask(torch, allowed))
    assert (got.parent == -1).all() and (got.next_parent == -1).all()


def test_beams_without_log_probabilities():
    """NaN, +inf, all -inf, a row of the lowest value; scores of -inf, NaN and +inf."""
    torch = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((8, 9001), generator=g, device="cuda")
    x[0, 8000] = math.nan
    x[1, 3] = math.inf
    x[2] = -math.inf
    x[3] = torch.finfo(torch.float32).min
    x[4, 1:] = -math.inf  # one candidate
    c = torch.tensor([[0, 0, 0, -3, -1, -math.inf, math.nan, math.inf]], device="cuda")
    got = _run(torch, x, c, 20)
    assert set(got.parent.unique().tolist()) <= {3, 4}


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("W,V,k", [(4, 5000, 9), (64, 64, 128), (64, 9000, 128), (2, 70000, 100)])
def test_ties(dtype, W, V, k):
    """All logits equal, the two zeros among them, all beams alike: beams and tokens in their order."""
    torch = need_gpu()
    x = torch.zeros((W, V), dtype=getattr(torch, dtype), device="cuda")
    x[:, ::3] = -0.0
    from gemm_decode_register_gb300 import ops

    got = ops.beam_select(x, torch.zeros((1, W), device="cuda"), k)
    order = [(0, i) if i < V else (i // V, i % V) for i in range(k)]
    assert got.parent[0].tolist() == [r for r, _ in order] and got.token[0].tolist() == [v for _, v in order]


def test_few_distinct_values():
    """Sorted rows, long runs of equal logits, one beam far ahead of the others."""
    torch = need_gpu()
    V, W = 30000, 8
    x = torch.arange(V, device="cuda").flip(0).repeat(W, 1).float() / 7000
    x[1] = x[1].flip(0)
    x[2] = torch.round(x[2])
    x[3] = torch.round(x[3] * 4) / 4
    c = torch.tensor([[-9.0, -9, -9, -9, -40, -40, -40, -9]], device="cuda")
    for k in (1, 8, 16, 128):
        _run(torch, x, c, k)
        _run(torch, x.bfloat16(), c, k)
    c[0, 7] = 100.0
    got = _run(torch, x, c, 128)
    assert (got.parent == 7).all()


def test_ends():
    """Every beam's best token ends it; k too small for W others; eos 0, the value of an empty place."""
    torch = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((6, 800), generator=g, device="cuda")
    x[:, 0] = 9.0
    c = torch.zeros((2, 3), device="cuda")
    for k in (1, 3, 4, 6):
        got = _run(torch, x, c, k, eos=0)
    assert (got.next_parent >= 0).all() and (got.next_token != 0).all()


def test_first_step():
    torch = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((2, 6000), generator=g, device="cuda").repeat_interleave(5, 0)
    c = torch.full((2, 5), -math.inf, device="cuda")
    c[:, 0] = 0
    got = _run(torch, x, c, 10)
    assert (got.parent == torch.tensor([[0], [5]], device="cuda")).all()


def test_repeats_graphs_streams_and_workspaces():
    """The same bits on every call, in a graph whose inputs change, on two streams at once, in a caller's workspace."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(8)
    B, W, V = 3, 4, 70001
    xs = [torch.randn((B * W, V), generator=g, device="cuda") * 3 for _ in range(3)]
    cs = [torch.randn((B, W), generator=g, device="cuda") for _ in range(3)]
    want = [_run(torch, x, c) for x, c in zip(xs, cs)]
    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(a, b))  # noqa: E731
    ws = ops.beam_select_workspace(B, W, V, 2 * W)
    ws.fill_(255)
    assert same(ops.beam_select(xs[0], cs[0], workspace=ws), want[0])
    x, c = xs[0].clone(), cs[0].clone()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        ops.beam_select(x, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        out = ops.beam_select(x, c)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        c.copy_(cs[i])
        graph.replay()
        assert same(out, want[i])
    sts = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for r in range(8):
        for i, s in enumerate(sts):
            with torch.cuda.stream(s):
                outs.append((i, ops.beam_select(xs[i], cs[i])))
    torch.cuda.synchronize()
    assert all(same(o, want[i]) for i, o in outs)


@pytest.mark.parametrize("B,W,V,k", [(32, 32, 140000, 128), (1100, 32, 1000, 128)])
def test_many_rows(B, W, V, k):
    """Several stretches for each of a thousand rows; lists that do not fit the stream's 16 MiB (the second)."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    assert (ops.raw_call("mx_beam_select_workspace_size", B, W, V, k) > 16 << 20) == (B == 1100)
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((B * W, V), generator=g, device="cuda", dtype=torch.bfloat16)
    c = torch.randn((B, W), generator=g, device="cuda")
    got = ops.beam_select(x, c, k)
    lse = torch.logsumexp(x.double(), 1)
    for b in (0, 13, B - 1):
        key = (c[b].double()[:, None] + x[b * W:(b + 1) * W].double() - lse[b * W:(b + 1) * W, None]).flatten()
        top = key.sort(descending=True, stable=True)
        assert torch.allclose(got.score[b].double(), top.values[:k], rtol=0, atol=OFF + 32 * 2.0 ** -24)
        assert (key[(got.parent[b].long() - b * W) * V + got.token[b].long()] >= top.values[k - 1] - 2 * OFF).all()
