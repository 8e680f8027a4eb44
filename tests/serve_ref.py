"""Plain references of the decode loop's operators, in 64 bits or whole numbers: the beams' selection, and a pool of pages
kept with lists."""
from __future__ import annotations

import math

import numpy as np


def beam_candidates(logits, scores, W, allowed=None):
    """Of each batch entry every candidate as (key, row, logit, token), in order.  logits [rows][V] and scores [rows] fp64
    (numpy), allowed bool [rows][V]."""
    out = []
    for b in range(len(scores) // W):
        found = []
        for r in range(b * W, (b + 1) * W):
            ok = np.ones(logits.shape[1], bool) if allowed is None else allowed[r]
            z = logits[r][ok]
            if not math.isfinite(scores[r]) or len(z) == 0 or np.isnan(z).any() or not math.isfinite(z.max()):
                continue
            top, log = z.max(), math.log(np.exp(z - z.max()).sum())
            for v in np.nonzero(ok & (logits[r] > -math.inf))[0]:
                found.append((scores[r] + ((logits[r][v] - top) - log), r, logits[r][v], int(v)))
        found.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
        out.append(found)
    return out


def check_beams(got, want, W, k, eos, off):
    """got: ops.Beams; want: beam_candidates; off: how far a key may be.  Where two beams' keys are closer than that
    either order is right, so places are compared by key there, and by token where nothing is near."""
    score, parent, token = (t.double().cpu().numpy() for t in got[:3])
    order = [(np.array([-c[0] for c in found]), np.array([c[1] for c in found])) for found in want]
    for b, found in enumerate(want):
        place = {(c[1], c[3]): c for c in found}
        seen = set()
        for i in range(k):
            if i >= len(found):
                assert (score[b, i], parent[b, i], token[b, i]) == (-math.inf, -1, 0), (b, i)
                continue
            key, row, logit, tok = found[i]
            here = (int(parent[b, i]), int(token[b, i]))
            assert here in place and here not in seen, (b, i, here)
            seen.add(here)
            tol = off + abs(key) * 2.0 ** -24
            assert abs(score[b, i] - place[here][0]) <= tol, (b, i)
            keys, rows = order[b]  # (keys ascend: whether another beam has a candidate that near)
            lo, hi = np.searchsorted(keys, -key - 2 * tol), np.searchsorted(keys, -key + 2 * tol, side="right")
            if (rows[lo:hi] != row).any():
                assert abs(place[here][0] - key) <= 2 * tol, (b, i)
            else:
                assert here == (row, tok), (b, i, here, found[i])
        # next: the first W of these that do not end
        going = [i for i in range(min(k, len(found))) if int(token[b, i]) != eos][:W]
        ns, np_, nt = (t.double().cpu().numpy()[b] for t in got[3:])
        for o in range(W):
            if o < len(going):
                i = going[o]
                assert (ns[o], np_[o], nt[o]) == (score[b, i], parent[b, i], token[b, i]), (b, o)
            else:
                assert (ns[o], np_[o], nt[o]) == (-math.inf, -1, 0), (b, o)


class Pool:
    """The pool as lists: references of each page, the stack of free pages."""

    def __init__(self, P):
        self.refs, self.free = [0] * P, list(range(P - 1, -1, -1))

    def remap(self, ps, table, lens, parent, keep, add):
        """Rows of pages and lengths of the new sequences, and the copies (source, destination, tokens)."""
        P = len(self.refs)
        pages = lambda n: -(-n // ps)  # noqa: E731
        new = []
        for s, p in enumerate(parent):
            n = lens[p] if p >= 0 else 0
            kept = n if keep is None else min(n, max(keep[s], 0))
            a = (add if p >= 0 else 0) if isinstance(add, int) else max(add[s], 0)
            new.append((kept, a, table[p][:pages(kept)] if p >= 0 else []))
        held = list(self.refs)
        for row, n in zip(table, lens):
            for q in row[:pages(n)]:
                held[q] -= 1
        # holders that do not write the page, and the sequences that do, in order
        still, writers = list(held), {}
        for s, (kept, a, row) in enumerate(new):
            for j, q in enumerate(row):
                if a > 0 and kept % ps and j == len(row) - 1:
                    writers.setdefault(q, []).append(s)
                else:
                    still[q] += 1
        need = 0
        for s, (kept, a, row) in enumerate(new):
            need += pages(kept + a) - pages(kept)
        stays = {q: w[0] for q, w in writers.items() if still[q] == 0}
        need += sum(len(w) for w in writers.values()) - len(stays)
        if need > len(self.free):
            return None
        copies, rows, fresh = [], [], []
        for s, (kept, a, row) in enumerate(new):
            row = list(row)
            if a > 0 and kept % ps and stays.get(row[-1]) != s:
                fresh.append(self.free.pop())
                copies.append((row[-1], fresh[-1], kept % ps))
                row[-1] = fresh[-1]
            while len(row) < pages(kept + a):
                fresh.append(self.free.pop())
                row.append(fresh[-1])
            rows.append(row)
        for q in range(P):
            refs = still[q] + (q in stays)
            if refs == 0 and self.refs[q] > 0:
                self.free.append(q)
            self.refs[q] = refs
        for q in fresh:
            self.refs[q] = 1
        return rows, [kept + a for kept, a, _ in new], copies

    def compact(self, ps, table, lens):
        P = len(self.refs)
        mine = [0] * P
        for row, n in zip(table, lens):
            for q in row[:-(-n // ps)]:
                mine[q] += 1
        U = sum(r > 0 for r in self.refs)
        holes = [q for q in range(U) if self.refs[q] == 0]
        moved = [q for q in range(U, P) if self.refs[q] > 0 and mine[q] == self.refs[q]]
        to = dict(zip(moved, holes))
        for a, b in to.items():
            self.refs[a], self.refs[b] = 0, self.refs[a]
        self.free = [q for q in range(P - 1, -1, -1) if self.refs[q] == 0]
        rows = [[to.get(q, q) for q in row[:-(-n // ps)]] for row, n in zip(table, lens)]
        return rows, [(a, b, ps) for a, b in to.items()]
