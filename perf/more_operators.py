"""Cases of the operators around a decode loop: the beams' selection over
the vocabulary (``beam``), forking, reserving and freeing pages of the
cache with the copies that come of it (``remap``), compacting the pool
(``compact``), and the product of 8-bit integers (``i8``).

With ``own`` false, ``run`` computes an operator in its plain form
(elementary torch operations); with ``own`` true it calls the package.
Hidden size 8192, N = 10240 and N = 28672 are those of the package's dense
projections, 8 heads of 128 its cache's; vocabularies are generic.
"""
import math
import random

import numpy as np
import torch

own = False

# ------------------------------------------------------------------ cases


def listed():
    return [
        # four beams of one request: launch latency
        dict(name="beam_one_request", op="beam", B=1, W=4, V=32000, k=8, eos=2, dtype="fp32", pad=0, mask=False, dead=0),
        # grammar-constrained beams: bit masks, some that allow nothing, dead beams, an odd vocabulary
        dict(name="beam_masked", op="beam", B=3, W=5, V=50001, k=11, eos=0, dtype="fp32", pad=7, mask=True, dead=2),
        # a serving batch, logits as the prefill GEMM writes them
        dict(name="beam_batch", op="beam", B=16, W=8, V=128000, k=16, eos=128, dtype="bf16", pad=0, mask=False, dead=0),
        # wide beams of many requests
        dict(name="beam_wide", op="beam", B=64, W=16, V=152000, k=32, eos=1, dtype="bf16", pad=64, mask=False, dead=0),
        # one request's beams after a step: a few tails copied, one layer's cache
        dict(name="remap_one_request", op="remap", kind="beam", B=1, W=4, ctx=611, page=16, Hkv=8, D=128, kv="bf16",
             layers=1),
        # a serving step: rejected drafts cut off, finished requests freed, new prompts let in; block-float cache, odd pages
        dict(name="remap_serving", op="remap", kind="serve", B=96, W=1, ctx=6000, page=24, Hkv=2, D=64, kv="mxfp8",
             layers=3),
        # wide beams over long contexts, several layers copied at once
        dict(name="remap_beams_long", op="remap", kind="beam", B=16, W=8, ctx=8000, page=16, Hkv=8, D=128, kv="bf16",
             layers=2),
        # a small block-float pool made dense again
        dict(name="compact_small", op="compact", B=7, ctx=700, page=32, Hkv=4, D=128, kv="mxfp8", layers=2, fill=0.7),
        # a pool of several GB after a day of requests
        dict(name="compact_large", op="compact", B=48, ctx=6000, page=64, Hkv=8, D=128, kv="bf16", layers=2, fill=0.5),
        # one token through the fused QKV projection
        dict(name="i8_token", op="i8", M=1, N=10240, K=8192, x="bf16", y="fp32"),
        # eight beams' logits: the vocabulary projection
        dict(name="i8_vocabulary", op="i8", M=8, N=128000, K=8192, x="fp32", y="fp32"),
        # a prompt through the up projection
        dict(name="i8_prompt", op="i8", M=4096, N=28672, K=8192, x="bf16", y="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["beam", "beam", "beam", "remap", "remap", "remap", "compact", "i8", "i8", "i8"])
    if op == "beam":
        W = _log_int(rng, 1, 32)
        V = _log_int(rng, 100, 160000)
        B = _log_int(rng, 1, max(1, min(64, 120_000_000 // (V * W))))
        return dict(op=op, B=B, W=W, V=V, k=rng.choice([W, 2 * W, 2 * W, 2 * W + rng.randint(0, 9)]),
                    eos=rng.choice([-1, 0, rng.randrange(V)]), dtype=rng.choice(["bf16", "fp32"]),
                    pad=rng.choice([0, 0, rng.randint(1, 64)]), mask=rng.random() < 0.4,
                    dead=rng.randint(0, W - 1) if rng.random() < 0.3 else 0)
    if op == "i8":
        K = 16 * _log_int(rng, 4, 1024)
        M = rng.choice([_log_int(rng, 1, 8), _log_int(rng, 1, 64), _log_int(rng, 1, 5000)])
        N = _log_int(rng, 40, max(41, min(160000, 1_000_000_000 // K, 900_000_000_000 // (M * K))))
        return dict(op=op, M=M, N=N, K=K, x=rng.choice(["bf16", "bf16", "fp32"]), y=rng.choice(["bf16", "fp32"]))
    c = dict(op=op, page=rng.choice([8, 16, 16, 32, 64, 48, 23]), Hkv=rng.randint(1, 8), D=rng.choice([64, 128]),
             kv=rng.choice(["bf16", "mxfp8"]), layers=rng.randint(1, 4))
    if op == "compact":
        c.update(B=rng.randint(1, 48), fill=rng.uniform(0.2, 0.95))
    else:
        c.update(kind=rng.choice(["beam", "serve"]))
        c.update(B=_log_int(rng, 1, 16), W=rng.randint(2, 8)) if c["kind"] == "beam" else c.update(B=_log_int(rng, 2, 128), W=1)
    # at most 3 GB of cache
    token = 2 * c["layers"] * c["Hkv"] * c["D"] * 2
    c["ctx"] = _log_int(rng, 40, max(41, min(8000, 3_000_000_000 // (3 * token * c["B"]))))
    return c


# ----------------------------------------------------------------- inputs


def _spread(lo, hi, B, first):
    """B whole numbers from lo to hi, the largest first, the others spread over the range."""
    return [hi if b == 0 else lo + int((hi - lo) * ((first + b * 0.6180339887498949) % 1.0)) for b in range(B)]


def _layout(case):
    """What the case says of the pool without its seed: logical pages of each slot (before the page numbers are dealt
    out), contexts, references, the step's parents, tokens to keep and to add."""
    page, S = case["page"], case["B"] * case.get("W", 1)
    rng = random.Random(case["ctx"] * 1000003 + S)
    slots, lens, refs = [], [], []

    def new(n):
        at = len(refs)
        refs.extend([1] * n)
        return list(range(at, at + n))

    parent, keep, add = list(range(S)), None, None
    if case.get("kind") == "beam":
        W = case["W"]
        for b, n in enumerate(_spread(max(1, case["ctx"] // 8), case["ctx"], case["B"], 0.3)):
            shared = new(int(n * rng.uniform(0.4, 0.95)) // page)  # the prompt's full pages, in all beams
            for w in range(W):
                if w:
                    for p in shared:
                        refs[p] += 1
                slots.append(shared + new(-(-n // page) - len(shared)))
                lens.append(n)
                parent[b * W + w] = b * W + int(W * rng.random() ** 2)  # good beams have several children
    else:
        common = new(case["ctx"] // (4 * page))  # a system prompt's pages, kept in a prefix cache too
        for n in _spread(1, case["ctx"], S, 0.3):
            mine = common[:n // page] if rng.random() < 0.5 else []
            for p in mine:
                refs[p] += 1
            slots.append(mine + new(-(-n // page) - len(mine)))
            lens.append(n)
        if case["op"] == "remap":
            keep, add = list(lens), [rng.randint(1, 6) for _ in range(S)]
            for s in range(S):
                u = rng.random()
                if u < 0.1:  # finished; a new prompt in its place or none
                    parent[s], add[s] = -1, rng.choice([0, rng.randint(1, case["ctx"])])
                elif u < 0.5:  # drafted tokens that were not accepted
                    keep[s] = max(0, lens[s] - rng.randint(1, 5))
    return slots, lens, refs, parent, keep, add


def _pool_pages(case, slots, refs):
    if case["op"] == "compact":
        return int(len(refs) / case["fill"]) + 1
    return len(refs) + len(slots) * (1 + -(-6 // case["page"])) + (case["ctx"] // case["page"] + 1) * (1 + len(slots) // 4) + 5


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    s = {"op": case["op"], "case": case}
    if case["op"] == "beam":
        return _prepare_beam(case, s, g)
    if case["op"] == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        x = randn(M, K)
        x[:, torch.randint(0, K, (1 + K // 500,), generator=g, device="cuda")] *= 12  # a few large channels
        s["x"] = x.to(torch.float32 if case["x"] == "fp32" else torch.bfloat16)
        s["w"] = (randn(N, K) * 40).round_().clamp_(-127, 127).to(torch.int8)
        s["w_scale"] = torch.exp(randn(N) * 0.3) * (0.02 / 40)
        return s
    slots, lens, refs, parent, keep, add = _layout(case)
    page, Hkv, D, layers = case["page"], case["Hkv"], case["D"], case["layers"]
    P, S = _pool_pages(case, slots, refs), len(slots)
    width = max(-(-(n + 8) // page) for n in lens + [case["ctx"]])
    order = torch.randperm(P, generator=g, device="cuda").int()  # page number of each logical page, then the free ones
    table = torch.full((S, width), -1, dtype=torch.int64)
    for i, pages in enumerate(slots):
        table[i, :len(pages)] = torch.tensor(pages, dtype=torch.int64)
    table = table.cuda()
    s["table"] = torch.where(table >= 0, order[table.clamp(min=0)], -1).int()
    s["table0"], s["table_out"] = s["table"].clone(), torch.zeros_like(s["table"])
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # pool: [free pages, 0, 0, 0], references of each page, the stack of free pages
    state = torch.zeros(4 + 2 * P, dtype=torch.int32, device="cuda")
    state[0] = P - len(refs)
    state[4 + order[:len(refs)].long()] = torch.tensor(refs, dtype=torch.int32, device="cuda")
    state[4 + P:4 + P + P - len(refs)] = order[len(refs):]
    s["state0"], s["state"], s["P"] = state, state.clone(), P
    if case["op"] == "remap":
        dev = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        s["parent"], s["keep"], s["add"] = dev(parent), dev(keep), dev(add)
    shape = (layers, P, Hkv, page, D)
    for half in "kv":
        if case["kv"] == "mxfp8":  # any finite codes, scales near one
            code = torch.randint(0, 127, shape, generator=g, device="cuda", dtype=torch.uint8)
            s[half] = code | (torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7)
            s[half + "_scales"] = torch.randint(118, 130, (*shape[:-1], D // 32), generator=g, device="cuda", dtype=torch.uint8)
        else:
            s[half] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
            s[half + "_scales"] = None
    if own:
        from gemm_decode_register_gb300 import ops

        s["pool"] = ops.PagePool(P, state=s["state"])
        s["layers"] = ops.PagedKVLayers([
            ops.PagedKV(s["k"][i], s["v"][i], s["table"],
                        *(None if s[h + "_scales"] is None else s[h + "_scales"][i] for h in "kv")) for i in range(layers)])
    return s


def _prepare_beam(case, s, g):
    B, W, V = case["B"], case["W"], case["V"]
    x = torch.randn((B * W, V + case["pad"]), generator=g, device="cuda") * 3
    s["logits"] = x.to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)[:, :V]
    c = torch.randn((B, W), generator=g, device="cuda") * 2 - 20  # log-probabilities of the beams so far
    if case["dead"]:
        c[0, W - case["dead"]:] = -math.inf
    s["scores"] = c
    s["mask"] = None
    if case["mask"]:
        n = (B * W, -(-V // 32))
        bits = lambda: torch.randint(-2 ** 31, 2 ** 31, n, generator=g, device="cuda").int()  # noqa: E731
        half, few = bits(), bits() & bits() & bits() & bits() & bits()
        kind = torch.randint(0, 4, (B * W, 1), generator=g, device="cuda")
        one = torch.zeros(n, dtype=torch.int32, device="cuda")
        one[:, V // 64] = 1  # a single token
        m = torch.where(kind == 0, half, torch.where(kind == 1, few, torch.where(kind == 2, one, -1)))
        m[B * W // 2] = 0  # a beam that may take none
        s["mask"] = m.int().contiguous()
    return s


# ------------------------------------------------------------ plain forms


def _beam(s):
    c = s["case"]
    B, W, V, k, eos = c["B"], c["W"], c["V"], c["k"], c["eos"]
    x = s["logits"].float() + 0.0  # (-0 becomes +0: the two are equal)
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        x = x.masked_fill((s["mask"][:, v >> 5] >> (v & 31)) & 1 == 0, -math.inf)
    top = x.amax(1, keepdim=True)
    # the sum over the vocabulary, and what is compared across beams, in 64 bits: near ties decide which beam wins
    lse = top[:, 0].double() + (x - top).exp().sum(1, dtype=torch.float64).log()
    # (logit, token) as one whole number: larger logits first, then lower tokens
    bits = x.view(torch.int32)
    bits = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long()
    n = min(k, V)
    best = ((bits << 32) | (0x7FFFFFFF - torch.arange(V, device="cuda"))).topk(n, dim=1).values
    token = 0x7FFFFFFF - (best & 0xFFFFFFFF)
    key = s["scores"].reshape(-1, 1).double() + (x.gather(1, token) - lse[:, None])
    key = torch.where(key.isfinite(), key, -math.inf).view(B, W * n)
    order = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    key = key.gather(1, order)
    token = token.view(B, W * n).gather(1, order)
    parent = order // n + torch.arange(B, device="cuda")[:, None] * W
    if key.shape[1] < k:
        more = (0, k - key.shape[1])
        key = torch.nn.functional.pad(key, more, value=-math.inf)
        token, parent = (torch.nn.functional.pad(t, more) for t in (token, parent))
    none = key == -math.inf
    out = {"score": key.float(), "parent": parent.masked_fill(none, -1).int(), "token": token.masked_fill(none, 0).int()}
    # the beams that go on: the first W that do not end
    ends = none | (token == eos)
    first = ends.int().sort(dim=1, stable=True).indices[:, :W]
    none = ends.gather(1, first)
    for name, rest in (("score", -math.inf), ("parent", -1), ("token", 0)):
        t = out[name].gather(1, first).masked_fill(none, rest)
        out["next_" + name] = torch.nn.functional.pad(t, (0, W - t.shape[1]), value=rest)
    return out


def _copy_pages(s, src, dst, tokens):
    """Pages dst[i] take the first tokens[i] tokens of pages src[i], in every layer and half."""
    part = torch.arange(s["case"]["page"], device="cuda") < tokens[:, None]
    for name in ("k", "v", "k_scales", "v_scales"):
        x = s[name]
        if x is not None:
            x[:, dst] = torch.where(part[None, :, None, :, None], x[:, src], x[:, dst])


def _remap(s):
    page, P = s["case"]["page"], s["P"]
    state = s["state"].copy_(s["state0"])
    count, refs, free = state[0].long(), state[4:4 + P].long(), state[4 + P:]
    table, lens = s["table"].long(), s["kv_len"].long()
    S, width = table.shape
    j = torch.arange(width, device="cuda")
    live = s["parent"] >= 0
    p = s["parent"].long().clamp(min=0)
    kept = torch.where(live, lens[p], 0)
    if s["keep"] is not None:
        kept = torch.minimum(kept, s["keep"].long())
    add = live.long() if s["add"] is None else s["add"].long()
    have, need = -(-kept // page), -(-(kept + add) // page)
    src = table[p]

    def tally(pages, where, sign):  # pages past P take what does not count
        n = torch.zeros(P + 1, dtype=torch.int64, device="cuda")
        n.index_add_(0, torch.where(where, pages, P).flatten(), torch.full((pages.numel(),), sign, device="cuda"))
        return n[:P]

    full = (kept // page)[:, None]
    partial = kept % page != 0
    grows = partial & (add > 0)
    used = (j < full) | ((j == full) & (partial & ~grows)[:, None])
    base = refs + tally(table, j < -(-lens // page)[:, None], -1) + tally(src, used, 1)
    tail = torch.where(grows, src.gather(1, full.clamp(max=width - 1))[:, 0], P)
    slot = torch.arange(S, device="cuda")
    first = torch.full((P + 1,), S, device="cuda").scatter_reduce_(0, tail, slot, "amin")
    base1 = torch.cat([base, base.new_ones(1)])
    stays = grows & (base1[tail] == 0) & (first[tail] == slot)
    copied = grows & ~stays
    after = base + ((base == 0) & (first[:P] < S)).long()
    start = have - copied.long()
    n_new = need - start
    off = n_new.cumsum(0) - n_new
    fresh = (j >= start[:, None]) & (j < need[:, None])
    taken = free[(count - 1 - off[:, None] - (j - start[:, None])).clamp(0, P - 1)]
    out = torch.where(j < start[:, None], src.int(), torch.where(fresh, taken, s["table_out"]))
    s["table_out"].copy_(out)
    gone = ((after == 0) & (refs > 0)).nonzero()[:, 0]
    after[taken[fresh].long()] = 1
    left = count - n_new.sum()
    free[left + torch.arange(len(gone), device="cuda")] = gone.int()
    state[0] = left + len(gone)
    state[4:4 + P] = after
    who = copied.nonzero()[:, 0]
    _copy_pages(s, tail[who], out[who, start[who]].long(), (kept % page)[who])
    return {"table": s["table_out"], "kv_len": (kept + add).int(), "state": state}


def _compact(s):
    page, P = s["case"]["page"], s["P"]
    state, table = s["state"].copy_(s["state0"]), s["table"].copy_(s["table0"])
    refs = state[4:4 + P]
    used = torch.arange(table.shape[1], device="cuda") < -(-s["kv_len"].long() // page)[:, None]
    mine = torch.zeros(P, dtype=torch.int64, device="cuda")
    mine.index_add_(0, table[used].long(), torch.ones_like(table[used], dtype=torch.int64))
    held = refs > 0
    low = torch.arange(P, device="cuda") < held.sum()
    src, dst = (~low & held & (mine == refs)).nonzero()[:, 0], (low & ~held).nonzero()[:, 0]
    n = min(len(src), len(dst))
    src, dst = src[:n], dst[:n]
    to = torch.arange(P, device="cuda", dtype=torch.int32)
    to[src] = dst.int()
    table.copy_(torch.where(used, to[table.long().clamp(min=0)], table))
    refs[dst] = refs[src]
    refs[src] = 0
    empty = (refs == 0).nonzero()[:, 0].flip(0)  # the lowest is taken first
    state[0] = len(empty)
    state[4 + P:4 + P + len(empty)] = empty.int()
    _copy_pages(s, src, dst, torch.full_like(src, page))
    return {"table": table, "state": state}


def _i8(s):
    x = s["x"].float()
    scale = x.abs().amax(1, keepdim=True) / 127
    q = torch.where(scale > 0, (x / scale).round().clamp(-127, 127), 0.0)
    y = (q @ s["w"].float().T) * scale * s["w_scale"]
    return y.to(torch.float32 if s["case"]["y"] == "fp32" else torch.bfloat16)


def _values(s):
    """The cache as the values it holds: bf16, or E4M3 elements and E8M0 scales."""
    if s["k_scales"] is None:
        return {"k": s["k"], "v": s["v"]}
    e4m3, e8m0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return {"k": s["k"].view(e4m3), "v": s["v"].view(e4m3),
            "k_scales": s["k_scales"].view(e8m0), "v_scales": s["v_scales"].view(e8m0)}


def run(s):
    c, op = s["case"], s["op"]
    if not own:
        if op == "beam":
            return _beam(s)
        if op == "i8":
            return _i8(s)
        return {**(_remap(s) if op == "remap" else _compact(s)), **_values(s)}
    from gemm_decode_register_gb300 import ops

    if op == "beam":
        return ops.beam_select(s["logits"], s["scores"], c["k"], eos=c["eos"], mask=s["mask"])._asdict()
    if op == "i8":
        return ops.i8_mm(s["x"], s["w"], s["w_scale"], out_dtype=torch.float32 if c["y"] == "fp32" else torch.bfloat16)
    s["state"].copy_(s["state0"])
    if op == "remap":
        kv_len, copies = ops.kv_remap(s["pool"], c["page"], s["table"], s["kv_len"], s["parent"], s["table_out"],
                                      add=1 if s["add"] is None else s["add"], keep=s["keep"])
        ops.kv_copy_pages(s["layers"], copies)
        return {"table": s["table_out"], "kv_len": kv_len, "state": s["state"], **_values(s)}
    s["table"].copy_(s["table0"])
    ops.kv_copy_pages(s["layers"], ops.kv_compact(s["pool"], c["page"], s["table"], s["kv_len"]))
    return {"table": s["table"], "state": s["state"], **_values(s)}


# -------------------------------------------------------------- the floor


def work(case):
    if case["op"] == "beam":
        rows, V = case["B"] * case["W"], case["V"]
        return {"bytes": rows * V * (4 if case["dtype"] == "fp32" else 2) + (rows * -(-V // 32) * 4 if case["mask"] else 0)
                + 4 * rows + 12 * case["B"] * (case["k"] + case["W"]), "flops": 4 * rows * V}
    if case["op"] == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * (4 if case["x"] == "fp32" else 2) + N * K + 4 * N + M * N * (4 if case["y"] == "fp32" else 2),
                "flops": 2 * M * N * K}
    slots, lens, refs, parent, keep, add = _layout(case)
    token = case["layers"] * 2 * case["Hkv"] * (case["D"] * 2 if case["kv"] == "bf16" else case["D"] + case["D"] // 32)
    page, entries = case["page"], sum(map(len, slots))
    if case["op"] == "compact":
        P, used = _pool_pages(case, slots, refs), len(refs)
        moved = page * int(used * (1 - used / P))  # on average
        return {"bytes": 4 * (2 * entries + 2 * P) + 2 * token * moved, "flops": entries}
    out = moved = 0
    tails = set()
    for s, p in enumerate(parent):
        n = 0 if p < 0 else (lens[p] if keep is None else min(keep[s], lens[p]))
        more = (p >= 0) if add is None else add[s]
        out += -(-(n + more) // page)
        if n % page and more:
            at = slots[p][n // page]
            if at in tails or refs[at] > 1:
                moved += n % page
            tails.add(at)
    return {"bytes": 4 * (entries + out) + 16 * len(refs) + 2 * token * moved, "flops": entries + out}


# ------------------------------------------------------ 64-bit definition


def _exact_beam(case, s):
    B, W, V, k, eos = (case[n] for n in ("B", "W", "V", "k", "eos"))
    got = {n: [] for n in ("score", "parent", "token", "next_score", "next_parent", "next_token")}
    for b in range(B):
        found = []
        for w in range(W):
            r = b * W + w
            z = s["logits"][r].double()
            if s["mask"] is not None:
                ok = np.unpackbits(s["mask"][r].cpu().numpy().view(np.uint8), bitorder="little")[:V].astype(bool)
                z[torch.from_numpy(~ok).to(z.device)] = -math.inf
            total = torch.logsumexp(z, 0)
            if not (math.isfinite(float(total)) and math.isfinite(float(s["scores"][b, w]))):
                continue
            v = torch.sort(z, descending=True, stable=True).indices[:k]
            v = v[z[v] > -math.inf]
            score = (s["scores"][b, w].double() + (z[v] - total)).tolist()
            found += [(-a, r, i, t) for i, (a, t) in enumerate(zip(score, v.tolist()))]
        found.sort()
        found = [(-a, r, t) for a, r, _, t in found[:k]]
        going = [f for f in found if f[2] != eos][:W]
        for name, rows, n in (("", found, k), ("next_", going, W)):
            rows = rows + [(-math.inf, -1, 0)] * (n - len(rows))
            for i, part in enumerate(("score", "parent", "token")):
                got[name + part].append([f[i] for f in rows])
    return {n: torch.tensor(v, dtype=torch.float64 if "score" in n else torch.int32, device="cuda") for n, v in got.items()}


def _exact_copies(s, got, copies):
    for name in ("k", "v", "k_scales", "v_scales"):
        if s[name] is not None:
            x = _values(s)[name].clone()
            raw = x if s["k_scales"] is None else x.view(torch.uint8)
            for a, b, n in copies:
                raw[:, b, :, :n] = (s[name])[:, a, :, :n]
            got[name] = x
    return got


def _exact_remap(case, s):
    page, P = case["page"], s["P"]
    table, out, lens = s["table"].tolist(), s["table_out"].tolist(), s["kv_len"].tolist()
    state = s["state0"].tolist()
    refs, free = state[4:4 + P], state[4 + P:4 + P + state[0]]
    parent = s["parent"].tolist()
    held = [r > 0 for r in refs]
    for pages, n in zip(table, lens):
        for j in range(-(-n // page)):
            refs[pages[j]] -= 1
    plan, writers = [], {}
    for i, p in enumerate(parent):
        n = 0 if p < 0 else lens[p]
        if s["keep"] is not None:
            n = min(n, int(s["keep"][i]))
        a = (0 if p < 0 else 1) if s["add"] is None else int(s["add"][i])
        pages = [] if p < 0 else table[p][:-(-n // page)]
        write = n % page != 0 and a > 0
        for q in pages[:-1] if write else pages:
            refs[q] += 1
        if write:
            writers.setdefault(pages[-1], []).append(i)
        plan.append((n, a, pages, write))
    keeps = {who[0] for q, who in writers.items() if refs[q] == 0}
    for i in keeps:
        refs[plan[i][2][-1]] = 1
    copies, stack, fresh = [], list(free), []
    for i, (n, a, pages, write) in enumerate(plan):
        row = list(pages)
        if write and i not in keeps:
            copies.append((row[-1], stack[-1], n % page))
            row[-1] = stack.pop()
            fresh.append(row[-1])
        while len(row) < -(-(n + a) // page):
            row.append(stack.pop())
            fresh.append(row[-1])
        out[i][:len(row)] = row
    back = [q for q in range(P) if held[q] and refs[q] == 0]
    for q in fresh:
        refs[q] = 1
    left = len(stack)
    rest = state[4 + P:]
    rest[left:left + len(back)] = back
    new = [left + len(back), 0, 0, 0] + refs + rest
    int32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    got = {"table": int32(out), "kv_len": int32([n + a for n, a, _, _ in plan]), "state": int32(new)}
    return _exact_copies(s, got, copies)


def _exact_compact(case, s):
    page, P = case["page"], s["P"]
    table, lens, state = s["table0"].tolist(), s["kv_len"].tolist(), s["state0"].tolist()
    refs, rest = state[4:4 + P], state[4 + P:]
    places = {}
    for i, n in enumerate(lens):
        for j in range(-(-n // page)):
            places.setdefault(table[i][j], []).append((i, j))
    used = sum(r > 0 for r in refs)
    holes = [q for q in range(used) if refs[q] == 0]
    movers = [q for q in range(used, P) if refs[q] > 0 and len(places.get(q, ())) == refs[q]]
    copies = []
    for a, b in zip(movers, holes):
        for i, j in places[a]:
            table[i][j] = b
        refs[b], refs[a] = refs[a], 0
        copies.append((a, b, page))
    empty = [q for q in reversed(range(P)) if refs[q] == 0]
    rest[:len(empty)] = empty
    int32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    got = {"table": int32(table), "state": int32([len(empty), 0, 0, 0] + refs + rest)}
    return _exact_copies(s, got, copies)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "beam":
        return _exact_beam(case, s)
    if case["op"] == "remap":
        return _exact_remap(case, s)
    if case["op"] == "compact":
        return _exact_compact(case, s)
    # codes as the quantisation defines them (an fp32 quotient, to the nearest even integer), then 64 bits
    amax = s["x"].abs().float().max(1).values
    scale = amax / 127.0
    codes = torch.round(torch.div(s["x"].float(), scale[:, None])).double()
    codes[scale == 0] = 0
    codes = codes.clamp(-127, 127)
    y = torch.empty((case["M"], case["N"]), dtype=torch.float64, device="cuda")
    for i in range(0, case["N"], 4096):
        y[:, i:i + 4096] = codes @ s["w"][i:i + 4096].double().T
    return y * (scale.double()[:, None] * s["w_scale"].double())
