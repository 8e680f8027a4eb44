"""The attention layer of examples/attention_layer.py, step by step: every token that is in the cache is the right one, and
every token's output is the layer's in 64 bits over the cache as it was written."""
import os
import runpy

import pytest

import attn_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")


def _cached(kv, half, b, m):
    """fp64 [Hkv][m][D] of a sequence's context, from the pages."""
    import torch

    pages = kv.block_table[b, :-(-m // kv.k.shape[2])].long()
    x, sc = (kv.k, kv.k_scales) if half == 0 else (kv.v, kv.v_scales)
    x = x.double() if sc is None else ref.mxfp8_values(x, sc)
    return torch.cat([x[p] for p in pages], 1)[:, :m]


@pytest.mark.parametrize("kv", ["bf16", "mxfp8"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (12, 4, 64)])
def test_every_token(kv, Hq, Hkv, D):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    hidden = 512
    layer = runpy.run_path(EXAMPLE)["AttentionLayer"](hidden, Hq, Hkv, D, 40, 16, 2, 20,
                                                      ops.KV_MXFP8 if kv == "mxfp8" else ops.KV_BF16)
    w_qkv = ops.dequant(layer.fmt, *layer.w_qkv, layer.n_qkv, hidden).double()
    w_out = ops.dequant(layer.fmt, *layer.w_out, hidden, Hq * D).double()
    freq, factor = ops.rope_frequencies(D, 500000.0, "banded", factor=8.0)
    g = torch.Generator(device="cuda").manual_seed(5)
    past = [[torch.zeros((0, Hkv, D), dtype=torch.float64, device="cuda") for _ in "kv"] for _ in range(2)]
    # cached tokens: the rows' and the cache's bf16 roundings, 2^-8 of an element each at most (the rotation keeps a pair's
    # length); MXFP8 instead of the second half a step of E4M3, 2^-4 of an element, or for what saturates (up to 512 of 448)
    # 64 / 512
    cached = 2.0 ** -7 if kv == "bf16" else 2.0 ** -3 + 2.0 ** -8
    # outputs: rows and queries move scores whose spread is below 8, softmax weights, attention output, result and what the
    # fp32 sums add: (2 * 8 + 4) 2^-8
    limit = 20 * 2.0 ** -8
    for new in ([70, 33], [1, 1], [0, 1], [5, 30], [1, 1], [1, 0]):
        start = layer.lens.copy()
        x = torch.randn((sum(new), hidden), generator=g, device="cuda").to(torch.bfloat16)
        y = layer(x, *layer.grow(new)).double()
        assert ops.device_error() == 0
        rows = (x.double() @ w_qkv.T).view(sum(new), -1, D)
        first = 0
        for b, n in enumerate(new):
            r = rows[first:first + n]
            pos = torch.arange(start[b], start[b] + n, device="cuda")
            qk = ref.rotate(r[:, :Hq + Hkv], pos, freq, factor)
            past[b][0] = torch.cat([past[b][0], qk[:, Hq:]])
            past[b][1] = torch.cat([past[b][1], r[:, Hq + Hkv:]])
            halves = [_cached(layer.kv, half, b, int(layer.lens[b])) for half in range(2)]
            for half, name in enumerate("kv"):
                want = past[b][half].transpose(0, 1)
                off = (halves[half] - want).norm(dim=-1) / want.norm(dim=-1)
                assert off.max() <= cached, f"step {new}, sequence {b}: {name} off by {float(off.max()):.3e}"
            if n:
                out, _, _, _ = ref.attend(qk[:, :Hq], *halves, D ** -0.5)
                want = out.reshape(n, -1) @ w_out.T
                off = (y[first:first + n] - want).norm(dim=-1) / want.norm(dim=-1)
                assert off.max() <= limit, f"step {new}, sequence {b}: outputs off by {float(off.max()):.3e}"
            first += n
