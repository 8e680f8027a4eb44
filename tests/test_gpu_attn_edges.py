"""Attention over the paged cache where shapes, masks and caches are unusual:
few tokens of wide groups."""
import pytest

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
