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
