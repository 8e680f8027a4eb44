"""One attention layer with block-float weights, as a model runs it: fused QKV
projection, append to the paged cache with the rotation on the way, attention
over the cache, output projection.  A prompt goes in as one chunk, then
every sequence of the batch grows by a token per step.

    python examples/attention_layer.py [--kv mxfp8] [--tokens 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gemm_decode_register_gb300 import FMT_MXFP4, ops, synth  # noqa: E402


class AttentionLayer:
    """Weights, rotation table and cache of one layer; hidden, Hq * D multiples of 32."""

    def __init__(self, hidden: int, Hq: int, Hkv: int, D: int, pages: int, page_size: int, max_seqs: int,
                 max_pages: int, kv_fmt: int = ops.KV_BF16, max_len: int = 8192, seed: int = 0, fmt: int = FMT_MXFP4):
        self.hidden, self.Hq, self.Hkv, self.D, self.page, self.fmt = hidden, Hq, Hkv, D, page_size, fmt
        self.n_qkv = (Hq + 2 * Hkv) * D

        def weight(N, K, s):
            codes, scales = synth.weights(fmt, N, K, s, exp_lo=118, exp_hi=120)
            return [torch.from_numpy(a.reshape(-1)).cuda() for a in (codes, scales)]

        self.w_qkv = weight(self.n_qkv, hidden, seed)
        self.w_out = weight(hidden, Hq * D, seed + 1)
        freq, factor = ops.rope_frequencies(D, 500000.0, "banded", factor=8.0)
        self.table = ops.rope_table(freq, max_len, factor)
        self.block_table = torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device="cuda")
        self.kv = ops.PagedKV.empty(pages, Hkv, page_size, D, self.block_table, kv_fmt)
        self.free = list(range(pages))
        self.lens = np.zeros(max_seqs, dtype=np.int64)

    def grow(self, new: list[int]) -> tuple[torch.Tensor, torch.Tensor]:
        """Pages for new[b] more tokens of each sequence; q_start and kv_len of the step."""
        for b, n in enumerate(new):
            have, need = -(-self.lens[b] // self.page), -(-(self.lens[b] + n) // self.page)
            for j in range(have, need):
                self.block_table[b, j] = self.free.pop()
            self.lens[b] += n
        q_start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        return q_start, torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def _project(self, w, x: torch.Tensor, N: int) -> torch.Tensor:
        # few rows stream the weights (fp32 out), many go to the tensor cores (bf16 out)
        return ops.qmv(self.fmt, *w, x, N) if x.shape[0] <= 16 else ops.qmm(self.fmt, *w, x, N)

    def __call__(self, x: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor) -> torch.Tensor:
        """x bf16 [T][hidden] of the step's new tokens -> [T][hidden] (fp32 for up to 16 tokens, else bf16)."""
        rows = self._project(self.w_qkv, x, self.n_qkv)
        q = ops.kv_append(self.kv, rows, q_start, kv_len, self.Hq, self.table)
        o = ops.paged_attn(self.kv, q, q_start, kv_len)
        return self._project(self.w_out, o.view(x.shape[0], -1), self.hidden)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--kv", choices=("bf16", "mxfp8"), default="bf16")
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args()
    layer = AttentionLayer(8192, 64, 8, 128, 256, 64, 3, 64, ops.KV_MXFP8 if a.kv == "mxfp8" else ops.KV_BF16)
    g = torch.Generator(device="cuda").manual_seed(0)

    def step(new: list[int]) -> torch.Tensor:
        x = torch.randn((sum(new), layer.hidden), generator=g, device="cuda").to(torch.bfloat16)
        return layer(x, *layer.grow(new))

    y = step([700, 40, 1300])  # three prompts in one chunk
    print(f"prompts of 700, 40 and 1300 tokens: output {tuple(y.shape)}, rms {y.float().pow(2).mean().sqrt():.4g}")
    for i in range(a.tokens):
        y = step([1, 1, 1])
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens for each: contexts {layer.lens.tolist()}, output {tuple(y.shape)}, "
          f"rms {y.float().pow(2).mean().sqrt():.4g}")
    assert ops.device_error() == 0


if __name__ == "__main__":
    main()
