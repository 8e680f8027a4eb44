"""Beam search over a small model as a decode loop runs it, without the host in its way: one attention layer with
block-float weights over a paged cache, a vocabulary projection in 8-bit integers, the selection over beams and vocabulary,
and the cache's pages forked, grown and freed with it.

    python examples/beam_search.py [--beams 4] [--tokens 12] [--kv mxfp8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from attention_layer import AttentionLayer  # noqa: E402

from gemm_decode_register_gb300 import ops  # noqa: E402


class BeamSearch:
    """B requests of W beams each; slot b * W + w is beam w of request b.  embed bf16 [V][hidden], the vocabulary
    projection int8 [V][hidden] with a scale for each token."""

    def __init__(self, layer: AttentionLayer, embed: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, B: int, W: int,
                 max_pages: int, eos: int):
        self.layer, self.embed, self.w, self.w_scales, self.B, self.W, self.eos = layer, embed, w, w_scales, B, W, eos
        kv = layer.kv
        self.pool = ops.PagePool(kv.k.shape[0])
        # the tables of this step and the next; a cache handle for each
        self.tables = [torch.zeros((B * W, max_pages), dtype=torch.int32, device="cuda") for _ in range(2)]
        self.kvs = [ops.PagedKV(kv.k, kv.v, t, kv.k_scales, kv.v_scales) for t in self.tables]
        self.kv_len = torch.zeros(B * W, dtype=torch.int32, device="cuda")
        self.one_each = torch.arange(B * W + 1, dtype=torch.int32, device="cuda")
        self.scores = torch.full((B, W), float("-inf"), device="cuda")
        self.scores[:, 0] = 0.0  # a request begins as one beam
        self.steps: list[ops.Beams] = []

    def _move(self, parent: torch.Tensor, add: int | torch.Tensor) -> None:
        """Every slot's context becomes its parent's and grows by `add`."""
        self.kv_len, copies = ops.kv_remap(self.pool, self.layer.page, self.tables[0], self.kv_len, parent, self.tables[1], add)
        ops.kv_copy_pages(self.kvs[1], copies)
        self.tables.reverse()
        self.kvs.reverse()
        self.layer.kv = self.kvs[0]

    def prompt(self, tokens: list[list[int]]) -> None:
        """The prompts of the requests, in beam 0 of each; the others are forked from it by the first step."""
        new = torch.zeros(self.B * self.W, dtype=torch.int32)
        new[::self.W] = torch.tensor([len(t) for t in tokens], dtype=torch.int32)
        self._move(torch.full((self.B * self.W,), -1, dtype=torch.int32, device="cuda"), new.cuda())
        q_start = torch.cat([torch.zeros(1, dtype=torch.int32), new.cumsum(0, dtype=torch.int32)])
        x = self.embed[torch.tensor(sum(tokens, []), device="cuda")]
        y = self.layer(x, q_start.cuda(), self.kv_len)
        last = (q_start[1:].long() - 1)[::self.W].repeat_interleave(self.W).cuda()
        self.hidden = (x[last] + y[last]).bfloat16()

    def step(self) -> torch.Tensor:
        """One token for every beam; returns the logits it was chosen from."""
        logits = ops.i8_mm(self.hidden, self.w, self.w_scales, out_dtype=torch.float32)
        beams = ops.beam_select(logits, self.scores, 2 * self.W, self.eos)
        self.steps.append(beams)
        self.scores = beams.next_score
        self._move(beams.next_parent, 1)
        x = self.embed[beams.next_token.view(-1)]
        self.hidden = (x + self.layer(x, self.one_each, self.kv_len)).bfloat16()
        return logits

    def beam(self, slot: int, upto: int | None = None) -> list[int]:
        """Tokens of a beam that goes on after the first `upto` steps."""
        out = []
        for beams in reversed(self.steps[:upto]):
            out.append(int(beams.next_token.view(-1)[slot]))
            slot = int(beams.next_parent.view(-1)[slot])
        return out[::-1]

    def finished(self, request: int) -> list[tuple[float, list[int]]]:
        """(score, tokens) of the hypotheses that ended, the best first."""
        found = []
        for i, beams in enumerate(self.steps):
            for score, parent, token in zip(*(t[request].tolist() for t in beams[:3])):
                if token == self.eos and parent >= 0:
                    found.append((score, self.beam(parent, i) + [token]))
        return sorted(found, reverse=True)


def model(hidden: int, V: int, Hq: int, Hkv: int, D: int, pages: int, page: int, kv_fmt: int, seed: int = 0):
    layer = AttentionLayer(hidden, Hq, Hkv, D, pages, page, 1, 1, kv_fmt, max_len=1024, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    embed = torch.randn((V, hidden), generator=g, device="cuda").bfloat16()
    w = torch.randint(-127, 128, (V, hidden), generator=g, device="cuda", dtype=torch.int8)
    return layer, embed, w, torch.full((V,), 2.0 / (73 * hidden ** 0.5), device="cuda")


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=12)
    ap.add_argument("--kv", choices=("bf16", "mxfp8"), default="bf16")
    a = ap.parse_args()
    V, B = 32000, 2
    parts = model(2048, V, 16, 4, 128, 256, 16, ops.KV_MXFP8 if a.kv == "mxfp8" else ops.KV_BF16)
    s = BeamSearch(*parts, B, a.beams, 64, eos=7)
    g = torch.Generator().manual_seed(0)
    s.prompt([torch.randint(0, V, (n,), generator=g).tolist() for n in (100, 37)])
    for _ in range(a.tokens):
        s.step()
    assert ops.device_error() == 0
    for b in range(B):
        print(f"request {b}: best beam {float(s.scores[b, 0]):.3f} {s.beam(b * a.beams)}, {len(s.finished(b))} ended")
    print(f"pages in use: {s.pool.num_pages - int(s.pool.count)}")


if __name__ == "__main__":
    main()
