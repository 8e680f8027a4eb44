"""Attention over the paged cache where shapes, masks and caches are unusual:
few tokens of wide groups."""
import math

import pytest

import attn_ref as ref
from gpu_util import need_gpu
from test_gpu_attn import FMTS, Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(32, 1), (33, 1), (40, 1), (84, 2), (43, 1), (48, 1), (64, 1), (65, 1), (128, 1)])
def test_few_tokens_of_wide_groups(fmt, D, Hq, Hkv):
    """Up to a handful of tokens whose rows fill one row tile (128 rows of token and query head), more than one, or one each:
    the queries come token by token or by whole tiles."""
    need_gpu()
    for n in ([1], [2], [3], [4], [5], [1, 3], [2, 2]):
        Batch(n, [x + 70 * i + 3 for i, x in enumerate(n)], Hq, Hkv, D, 16, fmt).check()
    Batch([4], [2500], Hq, Hkv, D, 64, fmt).check(window=1000)


@pytest.mark.parametrize("page", [16, 48])
def test_call_without_sequences_keeps_the_order(page):
    """Between a projection and the rotation of its rows a call whose rows belong to no sequence (a padded step): the rotation
    still waits for the projection.  Pages of 48 go by direct loads."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops, synth

    T, N, K = 2048, 8192, 4096
    codes, scales = (torch.from_numpy(x.reshape(-1)).cuda() for x in synth.weights(synth.FMT_MXFP4, N, K, 1))
    x = torch.randn((T, K), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
    table = ops.rope_table(ops.rope_frequencies(128)[0], T)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    b = Batch([2], [20], 8, 1, 128, page)
    b.q_start.zero_()
    rows, attn = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(b.q)
    want = ops.rope(ops.qmm(synth.FMT_MXFP4, codes, scales, x, N).view(T, -1, 128), pos, table)
    got = torch.empty_like(want)
    ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, out=attn)
    for _ in range(5):
        rows.zero_()
        torch.cuda.synchronize()
        ops.qmm(synth.FMT_MXFP4, codes, scales, x, N, rows)
        ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, out=attn)
        ops.rope(rows.view(T, -1, 128), pos, table, out=got)
        assert torch.equal(got, want)
    assert not attn.any() and ops.device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,page", [(128, 16), (64, 64), (128, 48), (128, 256)])
@pytest.mark.parametrize("n,m,window,missing", [
    ([40, 1], [300, 70], 0, -1),        # the last page: the chunk's first tokens do not need it
    ([300, 1], [300, 70], 0, 0.5),      # a prompt, a page in the middle
    ([300, 1], [700, 70], 40, 0.6),     # a window: neither earlier nor later tokens
    ([200, 1], [9000, 70], 0, -1),      # cut across the GPU
    ([3, 3], [5000, 2000], 1500, 0.7)])
def test_a_missing_page_spoils_the_rows_that_need_it(fmt, D, page, n, m, window, missing):
    """And no others, whichever kernel takes the call."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch(n, m, 8, 2, D, page, fmt)
    good, good_lse = b.check(window=window)
    pages = -(-m[0] // page)
    j = pages - 1 if missing == -1 else int(missing * pages)
    table = b.kv.block_table.clone()
    table[0, j] = -1
    kv = ops.PagedKV(b.kv.k, b.kv.v, table, b.kv.k_scales, b.kv.v_scales)
    out, lse = ops.paged_attn(kv, b.q, b.q_start, b.kv_len, window=window, return_lse=True)
    assert ops.device_error() == 0x4
    pos = torch.arange(m[0] - n[0], m[0], device="cuda")
    first = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
    need = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    need[:n[0]] = (first < (j + 1) * page) & (pos >= j * page)
    assert need.any()
    assert torch.isnan(out[need]).all() and torch.isnan(lse[need]).all()
    # the other rows may be summed again one by one: each within half a bf16 ulp and 2^-8 of the values of the definition
    first = 0
    for s in range(2):
        k, v = b.context(s)
        rows = slice(first, first + n[s])
        want, l, tol, ltol = ref.attend(b.q[rows].double(), k, v, D ** -0.5, True, window)
        keep = ~need[rows]
        ref.assert_within(out[rows][keep], want[keep], tol[keep], "out")
        ref.assert_within(lse[rows][keep], l[keep], ltol[keep], "lse")
        first += n[s]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,m", [([20] * 40, [2000] * 40), ([40, 3] * 10, [6000, 3000] * 10)])
def test_rows_computed_again_outlast_a_wait(fmt, n, m):
    """Rows that are computed again one by one (a NaN among the values of the last token, which the others may not see) take
    longer than the other warps' waits may, which stand before a CTA's next items: nobody gives up while they go on."""
    need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch(n, m, 16, 8, 128, 16, fmt)
    for s in range(len(n)):
        page, slot = b.place(s, m[s] - 1)
        b.kv.v[page, :, slot, 5] = math.nan if fmt == "bf16" else 0x7F
        b.halves[1][page, :, slot, 5] = math.nan
    ops.debug_qmm_stall(False, 1_000_000)
    try:
        b.check()
    finally:
        ops.debug_qmm_stall(False, 0)


def _put(b, half, s, pos, d, value, fmt="bf16"):
    """A value into the cache and its copy; MXFP8: a NaN only, as its code."""
    page, slot = b.place(s, pos)
    (b.kv.v if half else b.kv.k)[page, :, slot, d] = value if fmt == "bf16" else 0x7F
    b.halves[half][page, :, slot, d] = value


@pytest.mark.parametrize("D,n,m", [(128, [6], [150]), (64, [1, 40], [513, 200]), (128, [1], [3000]), (64, [70, 5], [2500, 2600])])
def test_kinds_of_values(D, n, m):
    """NaN, infinities of one sign and of both, and sums that overflow, among what all rows see, what some see, and in the same
    dimensions and others; small items, two row tiles and items cut across the GPU."""
    need_gpu()
    nan, inf = math.nan, math.inf
    for case in ([(3, 5, inf)], [(3, 5, inf), (9, 5, -inf)], [(3, 5, nan), (9, 5, inf), (2, 6, -inf)],
                 [(3, 5, inf), (-1, 5, nan)], [(3, 5, -inf), (-2, 9, inf), (-1, D - 1, nan)], [(3, 5, inf), (-1, 5, -inf)],
                 [(3, 0, nan), (-1, 0, inf)]):
        b = Batch(n, m, 8, 2, D, 16)
        for pos, d, value in case:
            _put(b, 1, 0, pos % m[0], d, value)
        b.check()
        b.check(window=30)
    # sums beyond the type in one dimension, an infinity in another, in both signs
    b = Batch(n, m, 8, 2, D, 16)
    for x in (b.kv.v, b.halves[1]):
        x[..., 7] = x[..., 7].abs() * 0 + 3e38
        x[..., 40] = x[..., 40].abs() * 0 - 3e38
    b.halves[1] = b.kv.v.double()
    b.check()
    _put(b, 1, 0, 3, 5, inf)
    b.check()


@pytest.mark.parametrize("fmt", FMTS)
def test_a_value_that_all_rows_see_costs_no_second_pass(fmt):
    """A NaN that every row sees makes the call at most fifty times as long, not a thousand."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch([256], [8192], 64, 8, 128, 64, fmt)

    def shortest():
        times = []
        for _ in range(4):
            e = [torch.cuda.Event(enable_timing=True) for _ in "ab"]
            e[0].record()
            ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len)
            e[1].record()
            torch.cuda.synchronize()
            times.append(e[0].elapsed_time(e[1]))
        return min(times[1:])

    clean = shortest()
    _put(b, 1, 0, 17, 5, math.nan, fmt)
    assert shortest() <= 50 * clean
    assert torch.isnan(ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len)[..., 5]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 48])
def test_first_columns_of_a_wider_table(fmt, page):
    """A server keeps one wide table: rows are as far apart as it is wide, and what lies past the view's columns is no page of
    the context."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch([2, 40, 1], [70, 100, 300], 8, 2, 128, page, fmt)
    want = b.check()[0]
    table = b.kv.block_table
    n = table.shape[1]
    wide = torch.full((3, n + 13), 1, dtype=torch.int32, device="cuda")
    wide[:, :n] = table
    halves = (b.kv.k, b.kv.v)
    scales = (b.kv.k_scales, b.kv.v_scales)
    kv = ops.PagedKV(*halves, wide[:, :n], *scales)
    assert torch.equal(ops.paged_attn(kv, b.q, b.q_start, b.kv_len), want)
    assert torch.equal(ops.paged_attn(ops.PagedKV(*halves, wide, *scales), b.q, b.q_start, b.kv_len), want)
    one = ops.PagedKV(*halves, wide[2:, :n], *scales)
    first = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    assert torch.equal(ops.paged_attn(one, b.q[42:], first, b.kv_len[2:]), want[42:])
    assert ops.device_error() == 0
    # a page of the last context is past the view: missing for the attention, and for the append
    short = ops.PagedKV(*halves, wide[:, :299 // page], *scales)
    out = ops.paged_attn(short, b.q, b.q_start, b.kv_len)
    assert ops.device_error() == 0x4
    assert torch.isnan(out[42]).all() and torch.equal(out[:42], want[:42])
    rows = torch.randn((b.T, 12 * 128), device="cuda")
    before = b.kv.k.clone()
    q = ops.kv_append(short, rows, b.q_start, b.kv_len, 8, None)
    assert ops.device_error() == 0x4
    assert torch.isnan(q[42]).all() and torch.isfinite(q[:42]).all()
    at, slot = b.place(2, 299)
    assert torch.equal(b.kv.k[at, :, slot].view(torch.uint8), before[at, :, slot].view(torch.uint8))
    for table in (wide[:1].expand(3, n + 13), wide.t()[:3]):
        with pytest.raises(ValueError):
            ops.PagedKV(*halves, table, *scales)


@pytest.mark.parametrize("fmt", FMTS)
def test_unused_slots(fmt):
    """Batches most of whose sequences have no new tokens: before, between and after the ones that do, whole and cut items."""
    need_gpu()
    for B, some in ((100, {0: (3, 40)}), (100, {99: (1, 3000)}), (300, {0: (1, 20), 33: (5, 9), 290: (40, 700)}),
                    (2000, {1: (1, 5000), 500: (2, 4000), 1800: (1, 100), 1999: (1, 9000)}),
                    (700, {i: (1, 1500 + i) for i in range(0, 700, 69)})):
        Batch([some.get(i, (0, 0))[0] for i in range(B)], [some.get(i, (0, 0))[1] for i in range(B)], 8, 2, 64, 16, fmt).check()


def test_unused_slots_cost_little():
    """One token in a batch of 4096 slots takes at most ten times as long as by itself, not fifty."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    def shortest(B):
        b = Batch([1] + [0] * (B - 1), [300] + [0] * (B - 1), 8, 1, 128, 16)
        graph = torch.cuda.CUDAGraph()  # the call by itself, without the host's part
        out, ws = torch.empty_like(b.q), ops.paged_attn_workspace(1, B, 8, 1, 128)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, out=out, workspace=ws)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(10):
                ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, out=out, workspace=ws)
        times = []
        for _ in range(4):
            e = [torch.cuda.Event(enable_timing=True) for _ in "ab"]
            e[0].record()
            graph.replay()
            e[1].record()
            torch.cuda.synchronize()
            times.append(e[0].elapsed_time(e[1]))
        return min(times[1:])

    one, many = shortest(1), shortest(4096)
    assert many <= 10 * one, (many, one)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,page", [(128, 16), (64, 48), (96, 16), (256, 7)])
def test_sums_near_the_types_largest(fmt, D, page):
    """Averages of values near the largest number are finite, whichever kernel takes the call: their sum is not formed."""
    torch = need_gpu()
    b = Batch([1, 9, 1], [400, 70, 1], 4, 2, D, page, fmt)
    for sign, d in ((1, 7), (-1, D - 1)):
        if fmt == "bf16":
            b.kv.v[..., d] = b.halves[1][..., d] = sign * 3e38
            b.halves[1] = b.kv.v.double()
        else:  # 384 * 2^119 in the block of the dimension
            block = slice(d // 32 * 32, d // 32 * 32 + 32)
            b.kv.v[..., block] = 0
            b.kv.v[..., d] = 0x7C if sign > 0 else 0xFC
            b.kv.v_scales[..., d // 32] = 119 + 127
            b.halves[1] = ref.mxfp8_values(b.kv.v, b.kv.v_scales)
    out, _ = b.check()
    assert torch.isfinite(out).all() and out[0, 0, 7] > 1e38 and out[0, 0, D - 1] < -1e38


def test_strides_of_dimensions_of_one():
    """A dimension of length one may have any stride: a single token, page, head or place."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    def odd(t):
        """The same elements; dimensions of one get a stride that nothing could use."""
        return torch.as_strided(t, t.shape, [s if n > 1 or i == t.dim() - 1 else 3
                                             for i, (n, s) in enumerate(zip(t.shape, t.stride()))])

    for fmt in (ops.KV_BF16, ops.KV_MXFP8):
        for Hq, Hkv, page in ((4, 1, 16), (4, 2, 16), (1, 1, 1)):
            D, table = 64, torch.zeros((1, 1), dtype=torch.int32, device="cuda")
            kv = ops.PagedKV.empty(1, Hkv, page, D, table, fmt)
            view = ops.PagedKV(odd(kv.k), odd(kv.v), odd(table), *(odd(s) for s in (kv.k_scales, kv.v_scales) if s is not None))
            one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
            rows = torch.randn((1, (Hq + 2 * Hkv) * D), device="cuda")
            turn = ops.rope_table(ops.rope_frequencies(D)[0], 4)
            q = ops.kv_append(kv, rows, one, one[1:], Hq, turn)
            want = ops.paged_attn(kv, q, one, one[1:])
            assert torch.equal(ops.kv_append(view, odd(rows), one, one[1:], Hq, turn), q)
            assert torch.equal(ops.paged_attn(view, odd(q), one, one[1:]), want)
            x = rows.view(1, -1, D)
            turned = ops.rope(x, one[:1], turn)
            out = torch.empty_like(x)
            assert torch.equal(ops.rope(odd(x), one[:1], turn, out=odd(out)), turned) and torch.equal(out, turned)
    assert ops.device_error() == 0


def test_windows_beyond_32_bits():
    """A window past the largest int is no window, not what is left of its bits; a negative one is refused."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    b = Batch([2], [40], 8, 1, 128, 16)
    want = b.check()[0]
    for window in ((1 << 31) - 1, 1 << 31, (1 << 32) + 5, (1 << 63) - 1, 1 << 64):
        assert torch.equal(ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, window=window), want)
    for window in (-1, 5 - (1 << 32)):
        with pytest.raises(ops.MxError):
            ops.paged_attn(b.kv, b.q, b.q_start, b.kv_len, window=window)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [1 << 20, (1 << 20) - 48])
@pytest.mark.parametrize("length", [(1 << 31) - 1, (1 << 31) - 127, (1 << 31) - 128])
def test_longest_contexts(fmt, page, length):
    """Contexts up to the largest int (a window over pages of which the last two exist): the end of the last key tile is past
    it.  Without the pages: NaN and the error, and the next call is right."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    D, n = 64, 3
    pages = (length - 1) // page + 1
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    table[0, -2:] = torch.tensor([1, 0], dtype=torch.int32)
    kv = ops.PagedKV.empty(2, 1, page, D, table, ops.KV_BF16 if fmt == "bf16" else ops.KV_MXFP8)
    for t in (kv.k, kv.v, kv.k_scales, kv.v_scales):
        if t is not None:
            t.fill_(math.nan if fmt == "bf16" else 0xFF)  # (0xFF: a NaN code, and the NaN scale)
    rows = torch.randn((300, 4 * D), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    first = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    kl = torch.tensor([length], dtype=torch.int32, device="cuda")
    q = ops.kv_append(kv, rows, first, kl, 2, None)[-n:].contiguous()
    first = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    at = torch.arange(length - 300, length, device="cuda")
    k, v = (h[table[0, at // page].long(), :, at % page].transpose(0, 1) for h in (
        (kv.k.double(), kv.v.double()) if fmt == "bf16" else
        (ref.mxfp8_values(kv.k, kv.k_scales), ref.mxfp8_values(kv.v, kv.v_scales))))
    for window in (1, 100, 280):
        out, lse = ops.paged_attn(kv, q, first, kl, window=window, return_lse=True)
        assert ops.device_error() == 0
        want, l, tol, ltol = ref.attend(q.double(), k, v, D ** -0.5, True, window)
        ref.assert_within(out, want, tol, "out")
        ref.assert_within(lse, l, ltol, "lse")
    table[0, -1] = -1
    out = ops.paged_attn(kv, q, first, kl, window=100)
    assert ops.device_error() == 0x4 and torch.isnan(out).all()
    Batch([1, 40], [9000, 300], 8, 1, 128, 64, fmt).check()
