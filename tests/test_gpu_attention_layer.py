"""The attention layer of examples/attention_layer.py (fused QKV projection,
append, attention, output projection with block-float weights) against the
same layer in 64 bits, over a prompt and the steps after it."""
import os
import runpy
import sys

import pytest

import attn_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")


@pytest.mark.parametrize("kv", ["bf16", "mxfp8"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (12, 4, 64)])
def test_layer(kv, Hq, Hkv, D):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    hidden = 512
    layer = runpy.run_path(EXAMPLE)["AttentionLayer"](hidden, Hq, Hkv, D, 40, 16, 2, 20,
                                                      ops.KV_MXFP8 if kv == "mxfp8" else ops.KV_BF16)
    w_qkv = ops.dequant(layer.fmt, *layer.w_qkv, layer.n_qkv, hidden).double()
    w_out = ops.dequant(layer.fmt, *layer.w_out, hidden, Hq * D).double()
    freq, factor = ops.rope_frequencies(D, 500000.0, "banded", factor=8.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    past = [[torch.zeros((0, Hkv, D), dtype=torch.float64, device="cuda") for _ in "kv"] for _ in range(2)]
    for new in ([70, 33], [1, 1], [1, 1], [5, 30], [1, 1]):
        start = layer.lens.copy()
        x = torch.randn((sum(new), hidden), generator=g, device="cuda").to(torch.bfloat16)
        y = layer(x, *layer.grow(new)).double()
        assert ops.device_error() == 0
        rows = (x.double() @ w_qkv.T).view(sum(new), -1, D)
        first, outs = 0, []
        for b, n in enumerate(new):
            r = rows[first:first + n]
            pos = torch.arange(start[b], start[b] + n, device="cuda")
            qk = ref.rotate(r[:, :Hq + Hkv], pos, freq, factor)
            past[b][0] = torch.cat([past[b][0], qk[:, Hq:]])
            past[b][1] = torch.cat([past[b][1], r[:, Hq + Hkv:]])
            out, _, _, _ = ref.attend(qk[:, :Hq], past[b][0].transpose(0, 1), past[b][1].transpose(0, 1), D ** -0.5)
            outs.append(out.reshape(n, -1))
            first += n
        want = torch.cat(outs) @ w_out.T
        # half ulps along the way: rows, queries, cache, weights of the softmax, attention output, result: six bf16 roundings
        # (2^-8 each at most), of which two move the scores, whose spread is below 8: (4 + 2 * 8) 2^-8; an MXFP8 cache
        # rounds keys and values to 2^-4 instead, root mean square 2^-5.8 at a mean mantissa: (1 + 8) 2^-5.8 more
        limit = 20 * 2.0 ** -8 + (9 * 2.0 ** -5.8 if kv == "mxfp8" else 0.0)
        rel = float((y - want).norm() / want.norm())
        assert rel <= limit, f"step {new}: relL2 {rel:.3e} > {limit:.3e}"


def test_example_runs(capsys, monkeypatch):
    need_gpu()
    monkeypatch.setattr(sys, "argv", [EXAMPLE, "--kv", "mxfp8", "--tokens", "3"])
    runpy.run_path(EXAMPLE, run_name="__main__")
    assert "contexts [703, 43, 1303]" in capsys.readouterr().out
