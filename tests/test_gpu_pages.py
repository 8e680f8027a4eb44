"""The page pool (mx_kv_remap, mx_kv_compact, mx_kv_copy_pages) against lists: every number after every step, and that every
sequence finds its tokens in its pages."""
import random

import pytest

import serve_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _i32(torch, v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _clean(pool):
    """The pool's own memory is as it was made: tallies, the word of faults, the bits of freed pages."""
    n, words = 8 * pool.num_pages, -(-pool.num_pages // 32) * 4
    return not bool(pool.work[:n + 4].any()) and not bool(pool.work[n + 16 + 64:n + 16 + 64 + words].any())


class Session:
    """A pool, a table and a cache whose tokens are numbers, next to the lists that say what should be there."""

    def __init__(self, torch, P, S, width, ps, wide=0):
        from gemm_decode_register_gb300 import ops

        self.torch, self.ops, self.P, self.S, self.ps = torch, ops, P, S, ps
        self.pool, self.ref = ops.PagePool(P), ref.Pool(P)
        self.tables = [torch.full((S, width + wide), -7, dtype=torch.int32, device="cuda")[:, :width] for _ in range(2)]
        self.rows, self.lens = [[] for _ in range(S)], [0] * S
        self.kv_len = _i32(torch, self.lens)
        self.text = [[] for _ in range(S)]
        self.kv = ops.PagedKV.empty(P, 1, ps, 8, self.tables[0])
        self.kv.k.zero_()
        self.kv.v.zero_()
        self.counter = 0

    def step(self, parent, keep=None, add=1):
        torch, ops = self.torch, self.ops
        want = self.ref.remap(self.ps, self.rows, self.lens, parent, keep, add)
        old = [self.tables[0].clone(), self.tables[1].clone(), self.pool.state.clone()]
        kv_len, copies = ops.kv_remap(self.pool, self.ps, self.tables[0], self.kv_len, _i32(torch, parent), self.tables[1],
                                      add if isinstance(add, int) else _i32(torch, add),
                                      None if keep is None else _i32(torch, keep))
        assert torch.equal(self.tables[0], old[0])
        if want is None:
            assert ops.device_error() == 0x10
            assert (kv_len == -1).all() and copies[0, 0] == 0
            assert torch.equal(self.tables[1], old[1]) and torch.equal(self.pool.state, old[2]) and _clean(self.pool)
            return False
        assert ops.device_error() == 0
        rows, lens, moves = want
        table = self.tables[1].tolist()
        assert kv_len.tolist() == lens
        for s, row in enumerate(rows):
            assert table[s][:len(row)] == row, s
            assert table[s][len(row):] == old[1][s, len(row):].tolist(), s
        assert copies[:1 + len(moves)].tolist() == [[len(moves), 0, 0, 0]] + [[*m, 0] for m in moves]
        ops.kv_copy_pages(self.kv, copies)
        kept = [(lens[s] - (add if p >= 0 else 0) if isinstance(add, int) else lens[s] - max(add[s], 0))
                for s, p in enumerate(parent)]
        self.text = [(self.text[p][:n] if p >= 0 else []) for p, n in zip(parent, kept)]
        self.rows, self.lens, self.kv_len = rows, lens, kv_len
        self.tables.reverse()
        for s in range(self.S):  # the new tokens
            for pos in range(kept[s], lens[s]):
                self.counter = self.counter % 200 + 1
                self.text[s].append(self.counter)
                self.kv.k[rows[s][pos // self.ps], 0, pos % self.ps] = self.counter
                self.kv.v[rows[s][pos // self.ps], 0, pos % self.ps] = -self.counter
        self.check()
        return True

    def compact(self):
        rows, moves = self.ref.compact(self.ps, self.rows, self.lens)
        copies = self.ops.kv_compact(self.pool, self.ps, self.tables[0], self.kv_len)
        self.ops.kv_copy_pages(self.kv, copies)
        assert self.ops.device_error() == 0
        assert copies[:1 + len(moves)].tolist() == [[len(moves), 0, 0, 0]] + [[*m, 0] for m in moves]
        table = self.tables[0].tolist()
        for s, row in enumerate(rows):
            assert table[s][:len(row)] == row, s
        self.rows = rows
        self.check()

    def check(self):
        n = int(self.pool.count)
        assert n == len(self.ref.free) and self.pool.free_pages[:n].tolist() == self.ref.free
        assert self.pool.refs.tolist() == self.ref.refs
        assert _clean(self.pool)
        k, v = self.kv.k[:, 0, :, 0].tolist(), self.kv.v[:, 0, :, 7].tolist()
        for s in range(self.S):
            at = [(self.rows[s][i // self.ps], i % self.ps) for i in range(self.lens[s])]
            assert [k[p][t] for p, t in at] == self.text[s], s
            assert [v[p][t] for p, t in at] == [-x for x in self.text[s]], s


@pytest.mark.parametrize("P,S,width,ps,seed", [(40, 1, 20, 4, 0), (64, 8, 12, 4, 1), (200, 5, 40, 1, 2), (300, 12, 200, 3, 3),
                                               (64, 16, 9, 16, 4), (3000, 90, 700, 2, 5), (33, 4, 30, 7, 6)])
def test_random_sessions(P, S, width, ps, seed):
    """Forks, cuts, ends, new prompts, growth by nothing or much, steps that the pool cannot supply, compaction."""
    torch = need_gpu()
    rng = random.Random(seed)
    t = Session(torch, P, S, width, ps, wide=3)
    full = 0
    for i in range(14):
        parent = [rng.choice([-1, s, s, s, rng.randrange(S)]) for s in range(S)]
        if i == 0:
            parent = [-1] * S
        keep = None if rng.random() < 0.4 else [rng.choice([10 ** 6, rng.randint(-1, 40)]) for _ in range(S)]
        room = max(1, P * ps // (2 * S))
        add = rng.choice([0, 1, 1, 3]) if rng.random() < 0.5 and i else [rng.randint(-1, room) for _ in range(S)]
        longest = max(t.lens) + (add if isinstance(add, int) else max(add))
        if longest > width * ps:
            keep = [min(k if keep else 10 ** 6, 5) for k in (keep or [5] * S)]
            add = 1
        if not t.step(parent, keep, add):
            full += 1
            t.step([s if s % 2 else -1 for s in range(S)], None, 0)
        if rng.random() < 0.4:
            t.compact()
    t.compact()
    t.step([-1] * S, None, 1)
    assert t.pool.refs.sum() == 0 and int(t.pool.count) == P


@pytest.mark.parametrize("W,ps", [(2, 16), (5, 4), (16, 1), (64, 8)])
def test_beam_steps(W, ps):
    """Beams of two requests, token by token, all from one of them now and then."""
    torch = need_gpu()
    rng = random.Random(W)
    t = Session(torch, 4000, 2 * W, 60, ps)
    assert t.step([-1] * (2 * W), None, [37 if s % W == 0 else 0 for s in range(2 * W)])
    assert t.step([s // W * W for s in range(2 * W)], None, 1)
    for i in range(20):
        b = [rng.randrange(W) if i % 5 == 4 else None for _ in range(2)]
        assert t.step([s // W * W + (int(W * rng.random() ** 2) if b[s // W] is None else b[s // W]) for s in range(2 * W)])


def test_other_holders():
    """A page that a prefix cache holds is copied before a sequence writes in it, is not freed, and does not move."""
    torch = need_gpu()
    t = Session(torch, 30, 2, 10, 4)
    t.step([-1, -1], None, [10, 3])
    for q in (t.rows[0][2], t.rows[0][0]):
        t.pool.refs[q] += 1
        t.ref.refs[q] += 1
    t.step([0, 1])
    t.step([-1, 1])
    held = [q for q in range(30) if t.ref.refs[q] > 0 and q not in t.rows[1]]
    assert len(held) == 2
    t.compact()
    assert all(t.ref.refs[q] == 1 for q in held)


def test_more_or_fewer_sequences():
    """table_out may have other rows and sizes than table."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    pool, r = ops.PagePool(50), ref.Pool(50)
    a = torch.zeros((1, 5), dtype=torch.int32, device="cuda")
    n, _ = ops.kv_remap(pool, 8, a.new_zeros((1, 1)), _i32(torch, [0]), _i32(torch, [-1]), a, _i32(torch, [21]))
    rows, lens, _ = r.remap(8, [[]], [0], [-1], None, [21])
    b = torch.zeros((7, 9), dtype=torch.int32, device="cuda")
    m, copies = ops.kv_remap(pool, 8, a, n, _i32(torch, [0] * 7), b, 2)
    rows, lens, moves = r.remap(8, rows, lens, [0] * 7, None, 2)
    assert m.tolist() == lens and copies.tolist()[1:1 + len(moves)] == [[*x, 0] for x in moves] and len(moves) == 6
    c = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    k, _ = ops.kv_remap(pool, 8, b, m, _i32(torch, [6, 3]), c, 0, keep=_i32(torch, [8, 23]))
    rows, lens, _ = r.remap(8, rows, lens, [6, 3], [8, 23], 0)
    assert k.tolist() == lens and [c[s, :len(x)].tolist() for s, x in enumerate(rows)] == rows
    assert pool.refs.tolist() == r.refs and pool.free_pages[:int(pool.count)].tolist() == r.free and _clean(pool)
    assert ops.device_error() == 0


@pytest.mark.parametrize("what,bit", [("parent", 0x20), ("page", 0x4), ("negative page", 0x4), ("long", 0x4), ("out", 0x4),
                                      ("refs", 0x4), ("pages", 0x10), ("count", 0x4), ("huge add", 0x4)])
def test_a_step_that_does_not_fit_changes_nothing(what, bit):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    t = Session(torch, 40, 6, 12, 4)
    t.step([-1] * 6, None, [9, 30, 1, 17, 4, 22])
    t.step([0, 1, 1, 3, 4, 1])
    table, kv_len, out = t.tables[0], t.kv_len, t.tables[1]
    parent, add = [0, 1, 1, 3, 3, 5], 1
    if what == "parent":
        parent[4] = 6
    elif what == "page":
        table[1, 2] = 60
    elif what == "negative page":
        table[5, 0] = -1
    elif what == "long":
        kv_len[2] = 12 * 4 + 1
    elif what == "out":
        out = out[:, :7]  # the longest have 31 tokens and get the 32nd: 8 pages
    elif what == "refs":
        t.pool.refs[table[4, 0].long()] = 0  # (sequence 4 ends)
    elif what == "pages":
        add = 17  # 4 pages each and 2 copies: 26 of the 20 that are free
    elif what == "count":
        t.pool.count.fill_(41)
    elif what == "huge add":
        add = 2 ** 31 - 1
    old = [x.clone() for x in (table, out, t.pool.state)]
    n, copies = ops.kv_remap(t.pool, 4, table, kv_len, _i32(torch, parent), out, add)
    assert ops.device_error() == bit
    assert (n == -1).all() and copies[0].tolist() == [0, 0, 0, 0]
    assert all(torch.equal(a, b) for a, b in zip(old, (table, out, t.pool.state))) and _clean(t.pool)
    if what in ("page", "negative page", "long"):
        copies = ops.kv_compact(t.pool, 4, table, kv_len)
        assert ops.device_error() == bit and copies[0].tolist() == [0, 0, 0, 0]
        assert torch.equal(old[0], table) and torch.equal(old[2], t.pool.state) and _clean(t.pool)


def test_large_table():
    """4096 sequences, rows of several thousand entries, 200,000 pages."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    P, S, ps = 200_000, 4096, 4
    rng = random.Random(1)
    pool, r = ops.PagePool(P), ref.Pool(P)
    a, b = (torch.zeros((S, 3100), dtype=torch.int32, device="cuda") for _ in range(2))
    add = [rng.randint(0, 60) for _ in range(S)]
    add[17] = 3099 * ps + 1
    n, _ = ops.kv_remap(pool, ps, a.new_zeros((1, 1)), _i32(torch, [0]), _i32(torch, [-1] * S), a, _i32(torch, add))
    rows, lens, _ = r.remap(ps, [[]], [0], [-1] * S, None, add)
    parent = [rng.choice([-1, s, rng.randrange(S), 17 if s % 500 == 0 else s]) for s in range(S)]
    keep = [rng.randint(0, 12000) if s % 3 == 0 else 10 ** 6 for s in range(S)]
    parent[17] = 5
    m, copies = ops.kv_remap(pool, ps, a, n, _i32(torch, parent), b, 0, _i32(torch, keep))
    rows, lens, moves = r.remap(ps, rows, lens, parent, keep, 0)
    m2, copies = ops.kv_remap(pool, ps, b, m, _i32(torch, list(range(S))), a, 1)
    rows, lens, moves = r.remap(ps, rows, lens, list(range(S)), None, 1)
    assert ops.device_error() == 0 and m2.tolist() == lens and int(copies[0, 0]) == len(moves) > 0
    assert copies[1:1 + len(moves)].tolist() == [[*x, 0] for x in moves]
    t = a.tolist()
    assert all(t[s][:len(row)] == row for s, row in enumerate(rows))
    assert pool.refs.tolist() == r.refs and pool.free_pages[:int(pool.count)].tolist() == r.free and _clean(pool)
    rows, moves = r.compact(ps, rows, lens)
    copies = ops.kv_compact(pool, ps, a, m2)
    assert copies[:1 + len(moves)].tolist() == [[len(moves), 0, 0, 0]] + [[*x, 0] for x in moves]
    t = a.tolist()
    assert all(t[s][:len(row)] == row for s, row in enumerate(rows))
    assert pool.refs.tolist() == r.refs and pool.free_pages[:int(pool.count)].tolist() == r.free and _clean(pool)


def _filled(torch, shape, dtype, g):
    if dtype is torch.uint8:
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=dtype)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("layers,P,Hkv,ps,D,major", [(1, 9, 1, 1, 32, "heads"), (2, 12, 3, 5, 64, "tokens"),
                                                     (3, 20, 8, 16, 128, "heads"), (9, 10, 2, 24, 96, "both"),
                                                     (1, 10, 5, 300, 256, "tokens"), (40, 8, 2, 8, 64, "heads")])
def test_copies(fmt, layers, P, Hkv, ps, D, major):
    """Both halves and their scales, whole pages and first tokens, heads or tokens first, both halves in one tensor."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    g = torch.Generator(device="cuda").manual_seed(layers)
    caches, kept = [], []
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")

    def half(width, dtype):
        if major == "tokens":
            return [_filled(torch, (P, ps, Hkv, width), dtype, g).transpose(1, 2) for _ in "kv"]
        if major == "both":
            x = _filled(torch, (P, 2, Hkv, ps, width), dtype, g)
            return [x[:, 0], x[:, 1]]
        return [_filled(torch, (P, Hkv, ps, width), dtype, g) for _ in "kv"]

    for _ in range(layers):
        data = half(D, torch.uint8 if fmt else torch.bfloat16)
        scales = half(D // 32, torch.uint8) if fmt else []
        caches.append(ops.PagedKV(*data, table, *scales))
        kept.append([(x, x.clone()) for x in data + scales])
    moves = [(0, 3, ps), (0, 4, max(1, ps // 2)), (2, 5, 1), (1, 6, 0), (1, 7, ps + 5)]
    copies = _i32(torch, [[len(moves), 0, 0, 0]] + [[*m, 0] for m in moves] + [[1, 2, ps, 0]] * 3)
    ops.kv_copy_pages(ops.PagedKVLayers(caches) if layers > 1 else caches[0], copies)
    for pairs in kept:
        for x, old in pairs:
            for a, b, n in moves:
                old[b, :, :n] = old[a, :, :n]
            assert torch.equal(x.view(torch.uint8) if fmt == 0 else x, old.view(torch.uint8) if fmt == 0 else old)
    assert ops.device_error() == 0


def test_copies_of_pages_that_are_not_there():
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    kv = ops.PagedKV.empty(4, 1, 8, 64, torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    kv.k.copy_(torch.arange(4, device="cuda").view(4, 1, 1, 1).expand(4, 1, 8, 64))
    kv.v.fill_(5)
    ops.kv_copy_pages(kv, _i32(torch, [[99, 0, 0, 0], [0, 4, 8, 0], [-1, 1, 8, 0], [3, 2, 8, 0]]))  # more said than there are
    assert ops.device_error() == 0x4
    assert kv.k[:, 0, 0, 0].tolist() == [0, 1, 3, 3]


def test_graph_of_a_step():
    """A captured step, replayed: tables, lengths and the pool move on with every replay."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    t = Session(torch, 100, 4, 12, 4)
    t.step([-1] * 4, None, [13, 2, 7, 0])
    a, b = t.tables
    parent, kv_len = _i32(torch, [0, 0, 2, 1]), t.kv_len.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        n, copies = ops.kv_remap(t.pool, 4, a, kv_len, parent, b, 1)
        ops.kv_copy_pages(t.kv, copies)
        a.copy_(b)
        kv_len.copy_(n)
    rows, lens = t.rows, t.lens
    for _ in range(9):
        graph.replay()
        rows, lens, _ = t.ref.remap(4, rows, lens, [0, 0, 2, 1], None, 1)
    torch.cuda.synchronize()
    assert kv_len.tolist() == lens and [a[s, :len(r)].tolist() for s, r in enumerate(rows)] == rows
    assert t.pool.refs.tolist() == t.ref.refs and t.pool.free_pages[:int(t.pool.count)].tolist() == t.ref.free
    assert ops.device_error() == 0 and _clean(t.pool)
