"""examples/beam_search.py: selection, forked pages and attention together.  Every step's choice is the one its logits
call for, and every beam's logits are those of its own tokens read as one prompt."""
import os
import runpy
import sys

import pytest

import serve_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.mark.parametrize("kv", ["bf16", "mxfp8"])
@pytest.mark.parametrize("B,W,V,page,lens", [(2, 3, 500, 16, (21, 9)), (1, 8, 3001, 32, (64,)), (3, 1, 100, 16, (5, 16, 40))])
def test_search(kv, B, W, V, page, lens):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    if EXAMPLES not in sys.path:
        sys.path.insert(0, EXAMPLES)
    m = runpy.run_path(os.path.join(EXAMPLES, "beam_search.py"))
    fmt = ops.KV_MXFP8 if kv == "mxfp8" else ops.KV_BF16
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, V, (n,), generator=g).tolist() for n in lens]
    s = m["BeamSearch"](*m["model"](512, V, 8, 2, 64, 120, page, fmt), B, W, 8, eos=5)
    s.prompt(prompts)
    scores, seen = s.scores.clone(), []
    for i in range(7):
        logits = s.step()
        want = ref.beam_candidates(logits.double().cpu().numpy(), scores.double().cpu().numpy().reshape(-1), W)
        ref.check_beams(s.steps[-1], want, W, 2 * W, 5, 2.0 ** -16)
        if i:  # the logits' beams are those chosen one step before
            seen.append([(logits[r].double(), prompts[r // W] + s.beam(r, i)) for r in range(B * W)])
        scores = s.scores.clone()
    assert ops.device_error() == 0
    # pages: as many references as table entries, none lost
    entries = [s.tables[0][r, :-(-int(n) // page)].tolist() for r, n in enumerate(s.kv_len)]
    refs = torch.zeros(120, dtype=torch.int32)
    for p in sum(entries, []):
        refs[p] += 1
    assert s.pool.refs.cpu().tolist() == refs.tolist() and int(s.pool.count) == int((refs == 0).sum())
    # The same tokens as one prompt: other kernels, and the roundings of rows, queries, cache, weights, attention, output
    # and hidden state fall differently: 2^-8 of a value each, in both (2 * 7 * 2^-8), and one step of the 8-bit codes, 1/254 of the
    # largest of a token's values, which is some 4 of their root mean square (2^-6); MXFP8: the cache's codes
    # of values that round differently are a step apart, 2^-3 of some of them.
    limit = 14 * 2.0 ** -8 + 2.0 ** -6 + (2.0 ** -4 if kv == "mxfp8" else 0.0)
    for rows in (seen[0], seen[-1]):
        for got, tokens in rows:
            one = m["BeamSearch"](*m["model"](512, V, 8, 2, 64, 120, page, fmt), 1, 1, 8, eos=5)
            one.prompt([tokens])
            want = one.step()[0].double()
            off = float((got - want).norm() / want.norm())
            assert off <= limit, off
