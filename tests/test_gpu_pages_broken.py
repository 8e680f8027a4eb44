"""Pools that are not in order: a step that would hand out a page that is in use, or none of the pool's, and a compaction that
would cover one, change nothing."""
import random

import pytest

from gpu_util import need_gpu
from test_gpu_pages import Session, _clean, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,S,width,ps,deep", [(40, 6, 12, 4, 0), (40, 6, 12, 4, 5), (9000, 30, 260, 4, 2100), (70000, 40, 900, 2, 1023)])
@pytest.mark.parametrize("bad", [-1, "P", 2 ** 31 - 1, -2 ** 31, "used"])
def test_free_pages_that_cannot_be_handed_out(P, S, width, ps, deep, bad):
    """Place `deep` of the pages that the step is to be handed holds a number outside the pool or a page that has references."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    t = Session(torch, P, S, width, ps)
    add = [min(width * ps // 4, 9 + 7 * s) for s in range(S)]
    assert t.step([-1] * S, None, add)
    more = [width * ps // 3 if deep > 50 else ps] * S
    need = sum(-(-(n + m) // ps) - -(-n // ps) for n, m in zip(t.lens, more))
    count = int(t.pool.count)
    assert deep < need <= count
    at = count - 1 - deep
    good = int(t.pool.free_pages[at])
    t.pool.free_pages[at] = {"P": P, "used": t.rows[3][0]}.get(bad, bad)
    old = [x.clone() for x in (t.tables[0], t.tables[1], t.pool.state)]
    ident = _i32(torch, range(S))
    n, copies = ops.kv_remap(t.pool, ps, t.tables[0], t.kv_len, ident, t.tables[1], _i32(torch, more))
    assert ops.device_error() == 0x4
    assert (n == -1).all() and copies[0].tolist() == [0, 0, 0, 0]
    assert all(torch.equal(a, b) for a, b in zip(old, (t.tables[0], t.tables[1], t.pool.state))) and _clean(t.pool)
    # a step that does not come to that place, and the whole one after it is put right
    n, _ = ops.kv_remap(t.pool, ps, t.tables[0], t.kv_len, ident, t.tables[1], 0)
    assert ops.device_error() == 0 and n.tolist() == t.lens
    t.pool.free_pages[at] = good
    assert t.step(list(range(S)), None, more)


@pytest.mark.parametrize("P,S,width,ps", [(60, 6, 12, 4), (70000, 90, 300, 2)])
def test_pages_of_fewer_references_than_entries_are_not_covered(P, S, width, ps):
    """A page in use whose references fell to nothing, or are fewer than its entries, is no free place."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    rng = random.Random(P)
    t = Session(torch, P, S, width, ps)
    assert t.step([-1] * S, None, [rng.randint(1, width * ps // 2) for _ in range(S)])
    assert t.step([s // 2 * 2 if s % 3 else -1 for s in range(S)], None, 0)  # (free places, shared pages)
    row = max(t.rows, key=len)
    for page, refs in ((row[0], 0), (row[0], t.ref.refs[row[0]] - 1), (row[-1], 0)):
        was = int(t.pool.refs[page])
        t.pool.refs[page] = refs
        old = [x.clone() for x in (t.tables[0], t.pool.state)]
        copies = ops.kv_compact(t.pool, ps, t.tables[0], t.kv_len)
        assert ops.device_error() == 0x4 and copies[0].tolist() == [0, 0, 0, 0]
        assert torch.equal(old[0], t.tables[0]) and torch.equal(old[1], t.pool.state) and _clean(t.pool)
        t.pool.refs[page] = was
    t.compact()


@pytest.mark.parametrize("P,S,width,ps", [(40, 6, 12, 4), (70000, 90, 300, 2)])
@pytest.mark.parametrize("room", [2, 1, 0])
def test_more_free_pages_than_pages(P, S, width, ps, room):
    """A count of free pages that leaves less room on the stack than the three pages that a step releases: nothing is written
    behind it."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    whole = torch.full((4 + 2 * P + 64,), -77, dtype=torch.int32, device="cuda")  # (the pool's numbers, and what lies behind)
    state = whole[:4 + 2 * P]
    state.copy_(ops.PagePool(P).state)
    pool, tables = ops.PagePool(P, state=state), [torch.zeros((S, width), dtype=torch.int32, device="cuda") for _ in range(2)]
    none, add = _i32(torch, [-1] * S), _i32(torch, [3 * ps if s == 1 else 1 for s in range(S)])
    n, _ = ops.kv_remap(pool, ps, tables[1], torch.zeros_like(none), none, tables[0], add)
    assert ops.device_error() == 0 and n.tolist() == add.tolist()
    freed = sorted(tables[0][1, :3].tolist())
    pool.count.fill_(P - room)
    ends = _i32(torch, [s if s != 1 else -1 for s in range(S)])
    n, _ = ops.kv_remap(pool, ps, tables[0], n, ends, tables[1], 0)
    assert ops.device_error() == 0x4 and int(pool.count) == P
    assert pool.free_pages[P - room:].tolist() == freed[:room] and (whole[4 + 2 * P:] == -77).all() and _clean(pool)
    assert (pool.refs[torch.tensor(freed, device="cuda")] == 0).all()
