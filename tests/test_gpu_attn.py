"""Attention over the paged cache against its definition in 64 bits: single
tokens, chunks and prompts, both cache formats, masks that leave rows
empty, and what lies in places that a row may not see."""
import math

import numpy as np
import pytest

import attn_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


class Batch:
    """A batch over a cache whose unused places hold NaN, whose unused table
    entries are out of range and whose pages are dealt out at random."""

    def __init__(self, n, m, Hq=8, Hkv=1, D=128, page=16, fmt="bf16", tokens_major=False, seed=0, spread=1.0):
        import torch

        from gemm_decode_register_gb300 import ops

        self.n, self.m, self.Hq, self.Hkv, self.D = n, m, Hq, Hkv, D
        g = torch.Generator(device="cuda").manual_seed(seed)
        counts = [-(-max(x, 0) // page) for x in m]
        P = sum(counts) + 2
        order = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).int()
        bt = torch.full((len(n), max(counts) + 1), 1 << 30, dtype=torch.int32)
        bt[:, 1::2] = -1
        at = 0
        for b, c in enumerate(counts):
            bt[b, :c] = order[at:at + c]
            at += c
        bt = bt.cuda()

        def shaped(t):
            return t.transpose(1, 2).contiguous().transpose(1, 2) if tokens_major else t

        used = torch.zeros((P, page), dtype=torch.bool, device="cuda")
        for b, c in enumerate(counts):
            for j in range(c):
                used[bt[b, j].long(), :max(0, min(page, m[b] - j * page))] = True
        self.halves = []
        store = []
        for _ in "kv":
            x = torch.randn((P, Hkv, page, D), generator=g, device="cuda") * spread
            if fmt == "mxfp8":
                r, e = ref.mxfp8_quantize(x.double())
                codes = r.float().to(torch.float8_e4m3fn).view(torch.uint8)
                scales = (e + 127).to(torch.uint8).view(P, Hkv, page, D // 32)
                codes = torch.where(used[:, None, :, None], codes, torch.full_like(codes, 0x7F))
                scales = torch.where(used[:, None, :, None], scales, torch.full_like(scales, 0xFF))
                codes, scales = shaped(codes), shaped(scales)
                self.halves.append(ref.mxfp8_values(codes, scales))
                store.append((codes, scales))
            else:
                b16 = x.to(torch.bfloat16)
                b16 = shaped(torch.where(used[:, None, :, None], b16, torch.full_like(b16, math.nan)))
                self.halves.append(b16.double())
                store.append((b16, None))
        self.kv = ops.PagedKV(store[0][0], store[1][0], bt, store[0][1], store[1][1])
        T = sum(n)
        self.T = T
        self.q = (2 * torch.randn((T, Hq, D), generator=g, device="cuda")).to(torch.bfloat16)
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(m, dtype=torch.int32, device="cuda")
        self.page = page

    def place(self, b, pos):
        """(page, slot) of a position of a sequence."""
        return int(self.kv.block_table[b, pos // self.page]), pos % self.page

    def context(self, b):
        import torch

        m = max(self.m[b], 0)
        pages = self.kv.block_table[b, :-(-m // self.page)].long()
        return [torch.cat([h[p] for p in pages], 1)[:, :m] if m else h[0, :, :0] for h in self.halves]

    def check(self, scale=None, causal=True, window=0, sinks=None, q=None):
        import torch

        from gemm_decode_register_gb300 import ops

        q = self.q if q is None else q
        true_scale = 1 / math.sqrt(self.D) if scale is None else scale
        out, lse = ops.paged_attn(self.kv, q, self.q_start, self.kv_len, scale=scale, causal=causal, window=window,
                                  sinks=sinks, return_lse=True)
        assert ops.device_error() == 0
        first = 0
        for b, (n, m) in enumerate(zip(self.n, self.m)):
            if n:
                k, v = self.context(b)
                rows = slice(first, first + n)
                if m >= n:
                    w, l, tol, ltol = ref.attend(q[rows].double(), k, v, true_scale, causal,
                                                 window, sinks)
                else:  # the first tokens sit before the context
                    w, l, tol, ltol = ref.attend(q[rows].double()[n - max(m, 0):], k, v,
                                                 true_scale, causal, window, sinks)
                    rows = slice(first + n - max(m, 0), first + n)
                    early = slice(first, rows.start)
                    if causal:
                        assert not out[early].any() and torch.isfinite(out[early]).all()
                        want = torch.full_like(lse[early], -math.inf) if sinks is None else sinks.expand_as(lse[early])
                        assert torch.allclose(lse[early], want, rtol=1e-6, atol=0)
                ref.assert_within(out[rows], w, tol, f"sequence {b}: out")
                ref.assert_within(lse[rows], l, ltol, f"sequence {b}: lse")
            first += n
        again = ops.paged_attn(self.kv, q, self.q_start, self.kv_len, scale=scale, causal=causal, window=window,
                               sinks=sinks)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)), "two calls differ"
        return out, lse


FMTS = ["bf16", "mxfp8"]
HEADS = [(128, 8, 1), (128, 64, 8), (64, 8, 2), (128, 1, 1), (128, 7, 1), (64, 12, 4), (128, 6, 2), (64, 48, 1)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_single_tokens(fmt, D, Hq, Hkv):
    """One new token per sequence: contexts of one token, around page and tile edges, and long ones."""
    need_gpu()
    m = [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000, 4097]
    Batch([1] * len(m), m, Hq, Hkv, D, 16, fmt).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [1, 7, 16, 32, 48, 64, 128, 256, 512])
def test_page_sizes(fmt, page):
    need_gpu()
    Batch([1, 3, 40], [700, 3, 530], 8, 2, 128, page, fmt).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [8, 32, 64, 80, 96, 112, 128, 160, 192, 256])
def test_head_sizes(fmt, D):
    need_gpu()
    if fmt == "mxfp8" and D % 32:
        pytest.skip("whole blocks only")
    Batch([1, 9], [200, 70], 4, 2, D, 16, fmt).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
@pytest.mark.parametrize("window", [0, 1, 100])
def test_chunks(fmt, D, Hq, Hkv, window):
    """Chunks of many lengths in one batch (some empty), whole prompts and chunks on top of a context."""
    torch = need_gpu()
    sinks = torch.randn(Hq, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda") * 2
    b = Batch([5, 0, 1, 16, 17, 33, 130, 1], [5, 40, 260, 300, 17, 161, 130, 1], Hq, Hkv, D, 32, fmt)
    b.check(window=window)
    b.check(window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_prompt(fmt, D):
    """A prompt of several tiles of queries and keys, all causal; then without the mask."""
    need_gpu()
    b = Batch([777, 300], [777, 1111], 8, 2, D, 64, fmt)
    b.check()
    b.check(causal=False)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_see_nothing(fmt):
    """Empty contexts, and more new tokens than context: zeros, and lse of -infinity or the sink."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch([3, 4, 140, 1], [0, 2, 5, 9], 8, 1, 128, 16, fmt)
    b.check()
    b.check(sinks=torch.linspace(-3, 3, 8, device="cuda"))
    b.check(window=1)
    out, lse = ops.paged_attn(b.kv, b.q, b.q_start, torch.tensor([-5, 0, 0, 0], dtype=torch.int32, device="cuda"),
                              return_lse=True)
    assert not out.any() and (lse == -math.inf).all() and ops.device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_strides(fmt):
    """Tokens-major pages, queries inside a wider row, another scale, large scores."""
    torch = need_gpu()
    b = Batch([4, 1, 50], [90, 300, 60], 8, 2, 128, 32, fmt, tokens_major=True)
    wide = torch.full((b.T, 8 * 128 + 256), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:64 + 1024] = b.q.view(b.T, -1)
    b.check(q=wide[:, 64:64 + 1024].unflatten(1, (8, 128)), scale=0.3)
    b.check(scale=-2.0)
    b.check(scale=0.0)


@pytest.mark.parametrize("n,m", [([6], [150]), ([1, 40], [513, 200])])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_values_that_a_row_may_not_see(n, m, value):
    """A NaN or an infinity among the values (or the keys) of a later token, or before a window, leaves every row that may
    not see it alone; rows that see it take it as the definition does."""
    torch = need_gpu()
    for half in (1, 0):
        b = Batch(n, m, 8, 1, 128, 16)
        s = len(n) - 1
        for pos in (m[s] - 1, m[s] - 3, 17):
            page, slot = b.place(s, pos)
            (b.kv.v if half else b.kv.k)[page, 0, slot, 5] = value
            b.halves[half][page, 0, slot, 5] = value
        b.check(window=30)
        if half:
            b.check()


def test_split_context():
    """A context long enough to be cut across the GPU, a single token and a few."""
    need_gpu()
    Batch([1], [40001], 8, 1, 128, 64).check()
    Batch([3, 1], [20011, 33], 16, 2, 64, 128, "mxfp8").check(window=15000)


def test_missing_pages():
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch([1, 1, 2], [100, 40, 300], 8, 1, 128, 16)
    good = b.check()[0]
    for entry in (-1, 1 << 20):
        table = b.kv.block_table.clone()
        table[1, 1] = entry
        kv = ops.PagedKV(b.kv.k, b.kv.v, table)
        out, lse = ops.paged_attn(kv, b.q, b.q_start, b.kv_len, return_lse=True)
        assert ops.device_error() == 0x4
        assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
        assert torch.equal(out[[0, 2, 3]], good[[0, 2, 3]])
    # a context that reaches past its row of the block table
    out = ops.paged_attn(b.kv, b.q, b.q_start, torch.tensor([100, 40, 5000], dtype=torch.int32, device="cuda"))
    assert ops.device_error() == 0x4
    assert torch.isnan(out[2:]).all() and torch.equal(out[:2], good[:2])


def test_rows_of_no_sequence_are_left_alone():
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch([2, 3], [70, 20], 8, 1, 128, 16)
    good = b.check()[0]
    q = torch.cat([b.q, b.q])
    out = torch.full_like(q, 3.0)
    ops.paged_attn(b.kv, q, b.q_start, b.kv_len, out=out)
    assert torch.equal(out[:5], good) and (out[5:] == 3).all()


def test_pages_past_32_bits():
    """A cache whose pages lie past 2^32 elements: 64-bit offsets."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    P, page, D = 300000, 64, 128
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 12 GB on the device")
    k = torch.empty((P, 2, page, D), dtype=torch.bfloat16, device="cuda")
    small = Batch([1, 5], [200, 130], 8, 2, D, page)
    table = small.kv.block_table.clone()
    used = small.kv.block_table
    for i in range(2):
        for j in range(-(-small.m[i] // page)):
            table[i, j] = P - 1 - int(used[i, j])
            k[table[i, j].long()] = small.kv.k[used[i, j].long()]
    # the values of the same pages: one tensor for both halves would hide a wrong base, so swap pages by one
    v = torch.empty_like(k)
    for i in range(2):
        for j in range(-(-small.m[i] // page)):
            v[table[i, j].long()] = small.kv.v[used[i, j].long()]
    out = ops.paged_attn(ops.PagedKV(k, v, table), small.q, small.q_start, small.kv_len)
    want = ops.paged_attn(small.kv, small.q, small.q_start, small.kv_len)
    assert torch.equal(out, want)
    rows = torch.randn((6, 12 * D), device="cuda")
    kv = ops.PagedKV(k, v, table)
    ops.kv_append(kv, rows, small.q_start, small.kv_len, 8, None)
    assert torch.equal(k[table[0, 199 // page].long(), 1, 199 % page],
                       rows[0, 9 * D:10 * D].to(torch.bfloat16))
    assert ops.device_error() == 0


def test_streams_and_graph():
    """Two streams at once, each with its own workspace, and a captured graph replayed with new lengths."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch([1, 2, 1], [9001, 3000, 77], 8, 1, 128, 64)
    want = b.check()[0]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out, ws = torch.empty_like(want), ops.paged_attn_workspace(b.T, 3, 8, 1, 128)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, out=out, workspace=ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, out=out, workspace=ws)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    b.kv_len[0] = 500
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len))
    assert not torch.equal(out, want)


def test_refusals():
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch([1], [20], 8, 2, 128, 16)
    with pytest.raises(ValueError):
        ops.paged_attn(b.kv, b.q.float(), b.q_start, b.kv_len)
    with pytest.raises(ValueError):
        ops.paged_attn(b.kv, b.q[..., :64], b.q_start, b.kv_len)
    with pytest.raises(ValueError):
        ops.paged_attn(b.kv, b.q, b.q_start.long(), b.kv_len)
    with pytest.raises(ValueError):
        ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len.cpu())
    with pytest.raises(ValueError):
        ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, sinks=torch.zeros(7, device="cuda"))
    with pytest.raises(ops.MxError):
        ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, window=-1)
    with pytest.raises(ValueError):
        ops.paged_attn(b.kv, b.q[:, :7], b.q_start, b.kv_len)  # 7 query heads over 2 cache heads
    with pytest.raises(ValueError):
        ops.PagedKV(b.kv.k, b.kv.v[:, :1], b.kv.block_table)
    with pytest.raises(ValueError):
        ops.PagedKV(b.kv.k, b.kv.v, b.kv.block_table.long())
    with pytest.raises(ValueError):
        ops.rope(torch.zeros((2, 3, 64), device="cuda", dtype=torch.float16), b.kv_len, torch.zeros((4, 32, 2)))
    assert ops.device_error() == 0


@pytest.mark.parametrize("n,m", [([1, 1], [20000, 300]), ([300, 1], [900, 5])])
def test_timeout_then_recovers(n, m):
    """Queries that never come (the test hook withholds their loads): the waits give up, the outputs are NaN, and the next
    calls (whose cut items count arrivals in the same words) are right."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch(n, m, 8, 1, 128, 64)
    good = b.check()[0]
    ops.debug_qmm_stall(True, 1_000_000)
    try:
        out, lse = ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, return_lse=True)
        assert ops.device_error() & 0x2
    finally:
        ops.debug_qmm_stall(False, 0)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    for _ in range(2):
        assert torch.equal(ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len), good)
    assert ops.device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_mxfp8_values_are_exact(D):
    """A context of one token gives its value back: every E4M3 code under every E8M0 scale, decoded exactly (rounded to bf16 only
    where the product has no bf16), NaN codes and the NaN scale included."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    scales = torch.arange(256, dtype=torch.uint8, device="cuda")
    B = 256 * 256 // D  # sequence b: codes (b D + d) % 256 under the scale b D // 256
    codes = (torch.arange(B * D, device="cuda") % 256).to(torch.uint8).view(B, 1, 1, D)
    sc = scales[(torch.arange(B, device="cuda") * D // 256)].view(B, 1, 1, 1).expand(B, 1, 1, D // 32).contiguous()
    page = 16
    k = torch.zeros((B, 1, page, D), dtype=torch.uint8, device="cuda")
    v = torch.full_like(k, 0x7F)
    ks = torch.full((B, 1, page, D // 32), 127, dtype=torch.uint8, device="cuda")
    vs = torch.full_like(ks, 255)
    v[:, :, :1], vs[:, :, :1] = codes, sc
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    q_start = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    q = torch.ones((B, 2, D), dtype=torch.bfloat16, device="cuda")
    out = ops.paged_attn(ops.PagedKV(k, v, table, ks, vs), q, q_start, one)
    assert ops.device_error() == 0
    # MXFP8 values in bf16: at most 4 significant bits, so only the range rounds; fp32 holds what overflows as infinity
    want = ref.mxfp8_values(v[:, 0, 0], vs[:, 0, 0]).to(torch.float32).to(torch.bfloat16)
    for h in range(2):
        got = out[:, h]
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got[~nan], want[~nan])


def test_large_windows_and_many_sequences():
    """A window of the largest size is no window; more sequences than a warp looks at in a round, some empty."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch([3, 40, 1], [2, 100, 300], 8, 1, 128, 16)
    assert torch.equal(b.check()[0], b.check(window=(1 << 31) - 1)[0])
    n = [i % 3 for i in range(75)]
    Batch(n, [x + 7 * i % 190 for i, x in enumerate(n)], 4, 2, 64, 16, "mxfp8").check()
    Batch([1] * 1100, [1 + i % 40 for i in range(1100)], 2, 1, 64, 16).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 16, 2), (64, 9, 3)])
@pytest.mark.parametrize("n,m", [([1], [1024]), ([1], [1025]), ([70], [2048]), ([70], [2049]),
                                 ([1, 40, 0, 300, 1], [1025, 2300, 7, 1700, 1]), ([1, 1, 1], [1000, 20, 6000])])
def test_whole_and_cut_items(fmt, D, Hq, Hkv, n, m):
    """Both sides of the lengths from which work is divided, and mixes of them."""
    torch = need_gpu()
    b = Batch(n, m, Hq, Hkv, D, 64, fmt)
    b.check()
    b.check(window=1100, sinks=torch.randn(Hq, device="cuda"))


@pytest.mark.parametrize("n,m", [([6], [1500]), ([1, 40], [2500, 2300])])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_values_that_a_row_of_a_cut_item_may_not_see(n, m, value):
    test_values_that_a_row_may_not_see(n, m, value)
