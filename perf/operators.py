"""Cases of the attention-side operators: rotary positions (``rope``), the
append to a paged key/value cache with the rotation on the way
(``kv_append``) and attention of new tokens over that cache
(``paged_attn``).

With ``own`` false, ``run`` computes an operator in its plain form
(elementary torch operations in 32 bits); with ``own`` true it calls the
package.  The head sizes are those of the package's fused QKV projection
(hidden 8192, N = 10240 = (64 + 8 + 8) heads of 128) and a head size of 64.
"""
import math

import torch

own = False

# ------------------------------------------------------------------ cases


def listed():
    return [
        # q and k heads of four single-token requests, far into long contexts: launch latency
        dict(name="rope_decode", op="rope", T=4, H=72, D=128, rot=128, interleaved=False, inverse=False,
             dtype="bf16", pos_max=131072, gap=1024, scaling="none"),
        # a prompt whose q heads sit in the rows of the fused projection; half of each head rotates, YaRN scaling
        dict(name="rope_prompt_partial", op="rope", T=4096, H=64, D=128, rot=64, interleaved=True, inverse=False,
             dtype="bf16", pos_max=65536, gap=2048, scaling="yarn"),
        # gradient of a training batch's q, odd token count, 64-wide heads
        dict(name="rope_gradient", op="rope", T=5003, H=64, D=64, rot=64, interleaved=False, inverse=True,
             dtype="fp32", pos_max=8192, gap=0, scaling="linear"),
        # four single-token requests: fp32 rows as mx_qmv writes them, small pages
        dict(name="append_decode", op="append", B=4, q_min=1, q_max=1, ctx_min=700, ctx_max=9000, Hq=64, Hkv=8, D=128,
             rot=128, interleaved=False, page=16, kv="bf16", dtype="fp32", scaling="banded"),
        # ragged batch of chunks, small heads, block-float cache
        dict(name="append_ragged", op="append", B=13, q_min=1, q_max=117, ctx_min=1, ctx_max=3001, Hq=14, Hkv=2, D=64,
             rot=64, interleaved=True, page=32, kv="mxfp8", dtype="bf16", scaling="none"),
        # a 4096-token prompt chunk: bf16 rows as mx_qmm writes them, block-float cache
        dict(name="append_prompt", op="append", B=1, q_min=4096, q_max=4096, ctx_min=4096, ctx_max=4096, Hq=64, Hkv=8,
             D=128, rot=128, interleaved=False, page=64, kv="mxfp8", dtype="bf16", scaling="none"),
        # one request early in its answer: launch latency
        dict(name="attn_token_short", op="attn", B=1, q_min=1, q_max=1, ctx_min=131, ctx_max=131, Hq=64, Hkv=8, D=128,
             page=16, kv="bf16", causal=True, window=0, sinks=False),
        # a serving batch of single tokens over contexts of many lengths
        dict(name="attn_tokens_batch", op="attn", B=64, q_min=1, q_max=1, ctx_min=517, ctx_max=8192, Hq=64, Hkv=8,
             D=128, page=64, kv="bf16", causal=True, window=0, sinks=False),
        # few requests with long contexts, block-float cache: the context is cut across the GPU
        dict(name="attn_tokens_long_mxfp8", op="attn", B=5, q_min=1, q_max=1, ctx_min=24001, ctx_max=65536, Hq=64,
             Hkv=8, D=128, page=64, kv="mxfp8", causal=True, window=0, sinks=False),
        # verification of a few drafted tokens each, sinks
        dict(name="attn_verify", op="attn", B=16, q_min=2, q_max=6, ctx_min=1000, ctx_max=16384, Hq=64, Hkv=8, D=128,
             page=32, kv="bf16", causal=True, window=0, sinks=True),
        # chunks and single tokens in one batch, 64-wide heads, sliding window, block-float cache
        dict(name="attn_mixed_window", op="attn", B=6, q_min=1, q_max=1500, ctx_min=300, ctx_max=7000, Hq=64, Hkv=8,
             D=64, page=64, kv="mxfp8", causal=True, window=1024, sinks=True),
        # a 4096-token chunk on top of 4096 cached tokens
        dict(name="attn_prompt", op="attn", B=1, q_min=4096, q_max=4096, ctx_min=8192, ctx_max=8192, Hq=64, Hkv=8,
             D=128, page=128, kv="bf16", causal=True, window=0, sinks=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "attn", "attn", "attn"])
    D = rng.choice([64, 128, 128])
    if op == "rope":
        H = rng.randint(1, 80)
        T = _log_int(rng, 1, max(2, 33_000_000 // (H * D)))
        return dict(op=op, T=min(T, 9000), H=H, D=D, rot=rng.choice([D, D, D // 2]),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4, dtype=rng.choice(["bf16", "fp32"]),
                    pos_max=_log_int(rng, 4000, 131072), gap=rng.choice([0, 1024, 2048]),
                    scaling=rng.choice(["none", "linear", "yarn", "banded"]))
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, Hq=Hkv * rng.choice([1, 3, 4, 7, 8]), Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]),
             kv=rng.choice(["bf16", "mxfp8"]))
    if op == "append":
        B = rng.randint(1, 24)
        q_max = _log_int(rng, 1, max(2, 4000 // B))
        ctx_max = _log_int(rng, 16, 9000) + q_max
        c.update(B=B, q_min=rng.randint(1, q_max), q_max=q_max, ctx_min=rng.randint(1, ctx_max), ctx_max=ctx_max,
                 rot=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.5,
                 dtype=rng.choice(["bf16", "fp32"]), scaling=rng.choice(["none", "linear", "yarn", "banded"]))
        return c
    kind = rng.choice(["tokens", "tokens", "verify", "chunks"])
    if kind == "chunks":
        B = rng.randint(1, 6)
        q_max = _log_int(rng, 20, 4000 // B)
        q_min = rng.randint(1, q_max)
        ctx_max = min(8192, q_max + _log_int(rng, 1, 8192 // B))
    else:
        B = _log_int(rng, 1, 64)
        q_max = 1 if kind == "tokens" else rng.randint(2, 8)
        q_min = rng.randint(1, q_max)
        ctx_max = max(16, _log_int(rng, 16, max(64, min(65536, 320_000 // B))))
    c.update(B=B, q_min=q_min, q_max=q_max, ctx_min=rng.randint(1, ctx_max), ctx_max=ctx_max, causal=True,
             window=rng.choice([0, 0, 0, _log_int(rng, 1, ctx_max)]), sinks=rng.random() < 0.3)
    return c


# ----------------------------------------------------------------- inputs


def _spread(lo, hi, B, first):
    """B whole numbers from lo to hi, the largest first, the others spread over the range."""
    return [hi if b == 0 else lo + int((hi - lo) * ((first + b * 0.6180339887498949) % 1.0)) for b in range(B)]


def _lengths(case):
    """New tokens and context (new tokens included) of each sequence."""
    q = _spread(case["q_min"], case["q_max"], case["B"], 0.3)
    ctx = _spread(case["ctx_min"], case["ctx_max"], case["B"], 0.7)
    return q, [max(a, b) for a, b in zip(q, ctx)]


def _frequencies(rot, scaling):
    """Radians per position of the rot / 2 pairs, and the factor on cos and sin: base 500000; "linear": positions
    stretched 4 times; "yarn": 16 times over 4096, with the ramp between 32 and 1 turns; "banded": 8 times over 8192,
    the fast bands unchanged, the slow ones divided, a blend between."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return f / 4, 1.0
    if scaling == "yarn":
        dim = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(500000.0))  # noqa: E731
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / 16 * ramp, 0.1 * math.log(16.0) + 1
    if scaling == "banded":
        turns = 8192 * f / (2 * math.pi)
        blend = ((turns - 1) / (4 - 1)).clamp(0, 1)
        return f * blend + f / 8 * (1 - blend), 1.0
    return f, 1.0


def _table(n, rot, scaling):
    f, mscale = _frequencies(rot, scaling)
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f.cuda()
    return torch.stack([angle.cos() * mscale, angle.sin() * mscale], -1).float()  # [n][rot / 2][2]


def _to_mxfp8(x):
    """Codes and scales of fp32 x [..., D]: per 32 elements one E8M0 scale 2^e, e = floor(log2(max |x|)) - 8, and the
    elements x / 2^e rounded to E4M3, saturated."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax == 0, -127, torch.frexp(amax).exponent - 9).clamp(min=-127).to(torch.int32)
    codes = (b * ((127 - e) << 23).view(torch.float32)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.reshape(x.shape).view(torch.uint8), (e + 127).to(torch.uint8)


def _from_mxfp8(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float()
    s = torch.exp2(scales.float() - 127.0)
    return (v.reshape(*v.shape[:-1], -1, 32) * s[..., None]).reshape(v.shape)


def _cache(case, g, need):
    """Pages [P][Hkv][page][D] of both halves of the cache filled with other tokens' values, and a block table that
    deals them out in a random order.  `need`: the contexts' lengths."""
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    counts = [-(-n // page) for n in need]
    P = sum(counts) + 3
    order = torch.randperm(P, generator=g, device="cuda").int()
    table = torch.zeros((case["B"], max(counts)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    s = {"table": table, "k_scales": None, "v_scales": None}
    for half in "kv":
        x = torch.randn((P, Hkv, page, D), generator=g, device="cuda", dtype=torch.bfloat16)
        if case["kv"] == "mxfp8":
            s[half], s[half + "_scales"] = _to_mxfp8(x.float())
        else:
            s[half] = x
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    s = {"op": case["op"], "case": case}
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        rows = randn(T, H * D + case["gap"]).to(dtype)
        s["x"] = rows[:, :H * D].view(T, H, D)  # the first heads of a wider row
        s["positions"] = torch.randint(0, case["pos_max"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["rope"] = _table(case["pos_max"], case["rot"], case["scaling"])
        return s
    q, ctx = _lengths(case)
    s["T"], s["Q"], s["L"] = sum(q), max(q), max(ctx)
    s["q_start"] = torch.tensor([0] + torch.tensor(q).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s.update(_cache(case, g, ctx))
    if case["op"] == "append":
        s["rows"] = randn(s["T"], (case["Hq"] + 2 * case["Hkv"]) * case["D"]).to(dtype)
        s["rope"] = _table(s["L"], case["rot"], case["scaling"])
    else:
        # twice a unit normal: scores spread enough that some keys count for much more than others
        s["q"] = (2 * randn(s["T"], case["Hq"], case["D"])).to(torch.bfloat16)
        s["sinks"] = randn(case["Hq"]) if case["sinks"] else None
    if own:
        from gemm_decode_register_gb300 import ops

        s["kv"] = ops.PagedKV(s["k"], s["v"], s["table"], s["k_scales"], s["v_scales"])
    return s


# ------------------------------------------------------------ plain forms


def _rotate(x, angles, rot, interleaved, inverse):
    """x fp32 [T][H][D], angles [T][rot / 2][2] (cos, sin): the first rot dimensions of each head rotated by pairs."""
    cos, sin = angles[:, None, :, 0], angles[:, None, :, 1]
    if inverse:
        sin = -sin
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _token_places(s):
    """Sequence of each token, its number within the sequence's new tokens, and its place in the context."""
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(s["q_start"], t, right=True) - 1
    i = t - s["q_start"][b]
    return b, i, s["kv_len"][b] - (s["q_start"][b + 1] - s["q_start"][b]) + i


def _append(s):
    c = s["case"]
    T, Hq, Hkv, D, page = s["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    b, _, pos = _token_places(s)
    x = s["rows"].float().view(T, Hq + 2 * Hkv, D)
    turned = _rotate(x[:, :Hq + Hkv], s["rope"][pos], c["rot"], c["interleaved"], False)
    page_of, slot = s["table"][b, pos // page].long(), pos % page
    for half, new in (("k", turned[:, Hq:]), ("v", x[:, Hq + Hkv:])):
        if c["kv"] == "mxfp8":
            codes, scales = _to_mxfp8(new)
            s[half][page_of, :, slot] = codes
            s[half + "_scales"][page_of, :, slot] = scales
        else:
            s[half][page_of, :, slot] = new.to(torch.bfloat16)
    return turned[:, :Hq].to(torch.bfloat16)


def _context(s, half):
    """One half of the cache in context order, fp32 [B][Hkv][L][D]."""
    c = s["case"]
    x = s[half][s["table"].long()]  # [B][pages][Hkv][page][D]
    x = _from_mxfp8(x, s[half + "_scales"][s["table"].long()]) if c["kv"] == "mxfp8" else x.float()
    return x.transpose(1, 2).reshape(c["B"], c["Hkv"], -1, c["D"])[:, :, :s["L"]]


def _attend(s):
    c = s["case"]
    B, Q, L, Hq, Hkv, D = c["B"], s["Q"], s["L"], c["Hq"], c["Hkv"], c["D"]
    g = Hq // Hkv
    n_q = s["q_start"][1:] - s["q_start"][:-1]
    at = (s["q_start"][:-1, None] + torch.arange(Q, device="cuda")).clamp(max=s["T"] - 1)
    q = s["q"][at].float().view(B, Q, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * Q, D)
    score = torch.matmul(q, _context(s, "k").transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, g, Q, L)
    key = torch.arange(L, device="cuda")
    pos = (s["kv_len"] - n_q)[:, None] + torch.arange(Q, device="cuda")  # [B][Q]
    hidden = (key > pos[..., None]) | (key >= s["kv_len"][:, None, None])
    if c["window"]:
        hidden |= key <= pos[..., None] - c["window"]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(Hkv, g, 1, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + (sink - top).exp()
    out = torch.matmul(p.view(B, Hkv, g * Q, L), _context(s, "v")).view(B, Hkv, g, Q, D)
    out = torch.where(total == 0, 0.0, out / total)
    lse = (top + total.log())[..., 0]
    b, i, _ = _token_places(s)
    out = out.permute(0, 3, 1, 2, 4)[b, i].reshape(-1, Hq, D)
    return out.to(torch.bfloat16), lse.permute(0, 3, 1, 2)[b, i].reshape(-1, Hq).contiguous()


def _cache_values(s):
    """The cache as the values it holds: bf16, or E4M3 elements and E8M0 scales."""
    if s["k_scales"] is None:
        return {"k": s["k"], "v": s["v"]}
    e4m3, e8m0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return {"k": s["k"].view(e4m3), "v": s["v"].view(e4m3),
            "k_scales": s["k_scales"].view(e8m0), "v_scales": s["v_scales"].view(e8m0)}


def run(s):
    c = s["case"]
    if own:
        from gemm_decode_register_gb300 import ops

        if s["op"] == "rope":
            return ops.rope(s["x"], s["positions"], s["rope"], interleaved=c["interleaved"], inverse=c["inverse"])
        if s["op"] == "append":
            q = ops.kv_append(s["kv"], s["rows"], s["q_start"], s["kv_len"], c["Hq"], s["rope"],
                              interleaved=c["interleaved"])
            return {"q": q, **_cache_values(s)}
        out, lse = ops.paged_attn(s["kv"], s["q"], s["q_start"], s["kv_len"], causal=c["causal"], window=c["window"],
                                  sinks=s["sinks"], return_lse=True)
        return {"out": out, "lse": lse}
    if s["op"] == "rope":
        x = s["x"]
        y = _rotate(x.float(), s["rope"][s["positions"].long()], c["rot"], c["interleaved"], c["inverse"])
        return y.to(x.dtype)
    if s["op"] == "append":
        return {"q": _append(s), **_cache_values(s)}
    out, lse = _attend(s)
    return {"out": out, "lse": lse}


# -------------------------------------------------------------- the floor


def work(case):
    D = case["D"]
    e = 4 if case.get("dtype") == "fp32" else 2
    if case["op"] == "rope":
        T, H = case["T"], case["H"]
        return {"bytes": T * (2 * H * D * e + 4 + 4 * case["rot"]), "flops": 3 * T * H * case["rot"]}
    q, ctx = _lengths(case)
    T, Hq, Hkv = sum(q), case["Hq"], case["Hkv"]
    row = D * 2 if case["kv"] == "bf16" else D + D // 32  # one head of one cached token, one half
    if case["op"] == "append":
        return {"bytes": T * ((Hq + 2 * Hkv) * D * e + 4 * case["rot"] + Hq * D * 2 + 2 * Hkv * row),
                "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    pairs = keys = 0
    for n, m in zip(q, ctx):
        w = case["window"] or m
        keys += min(m, w + n - 1)
        pairs += sum(min(w, m - n + i + 1) for i in range(n))
    return {"bytes": 2 * T * Hq * D * 2 + T * Hq * 4 + 2 * keys * Hkv * row, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------ 64-bit definition


def _exact_turn(x, pos, rot, interleaved, inverse, scaling):
    """x fp64 [T][H][D] turned pair by pair, as complex numbers."""
    f, mscale = _frequencies(rot, scaling)
    angle = pos.double()[:, None] * f.to(pos.device)
    turn = torch.polar(torch.full_like(angle, mscale), -angle if inverse else angle)[:, None]
    y = x.clone()
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_cached(s, half, pages):
    """fp64 values of some pages, [n][Hkv][page][D], E4M3 decoded from its bits."""
    x = s[half][pages]
    if s[half + "_scales"] is None:
        return x.double()
    code = torch.arange(256)
    field, frac = (code >> 3) & 15, (code & 7).double()
    value = torch.where(field == 0, frac * 2.0 ** -9, (8 + frac) * 2.0 ** (field.double() - 10))
    value = torch.where(code >= 128, -value, value).to(x.device)
    scale = 2.0 ** (s[half + "_scales"][pages].double() - 127)
    return value[x.long()] * scale.repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(s["x"].double(), s["positions"], case["rot"], case["interleaved"], case["inverse"],
                           case["scaling"])
    n_q, ctx = _lengths(case)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "append":
        mx = case["kv"] == "mxfp8"
        pos = torch.tensor([m - n + i for n, m in zip(n_q, ctx) for i in range(n)], device="cuda")
        seq = torch.tensor([b for b, n in enumerate(n_q) for _ in range(n)], device="cuda")
        x = s["rows"].double().view(s["T"], -1, D)
        turned = _exact_turn(x[:, :Hq + Hkv].contiguous(), pos, case["rot"], case["interleaved"], False,
                             case["scaling"])
        at = s["table"][seq, pos // page].long()
        got = {"q": turned[:, :Hq]}
        for half, new in (("k", turned[:, Hq:]), ("v", x[:, Hq + Hkv:])):
            old = s[half].view(torch.float8_e4m3fn) if mx else s[half]
            got[half] = old.double()
            if mx:  # the elements before their rounding, cut at the largest, over the block's power of two
                blocks = new.reshape(s["T"], Hkv, D // 32, 32)
                e = torch.floor(torch.log2(blocks.abs().amax(-1))) - 8
                got[half + "_scales"] = 2.0 ** (s[half + "_scales"].double() - 127)
                got[half + "_scales"][at, :, pos % page] = 2.0 ** e
                new = (blocks / 2.0 ** e[..., None]).clamp(-448, 448).reshape(s["T"], Hkv, D)
            got[half][at, :, pos % page] = new
        return got
    pairs = work(case)["flops"]
    if pairs > 4e12:
        return None
    out = torch.zeros((s["T"], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, m) in enumerate(zip(n_q, ctx)):
        pages = s["table"][b, :-(-m // page)].long()
        k, v = (_exact_cached(s, half, pages).transpose(0, 1).reshape(Hkv, -1, D)[:, :m] for half in "kv")
        for h in range(Hq):
            for i in range(0, n, 1024):
                t = torch.arange(i, min(n, i + 1024), device="cuda")
                here = (m - n + t)[:, None]
                key = torch.arange(m, device="cuda")
                seen = (key <= here) & ((key > here - case["window"]) if case["window"] else (key >= 0))
                z = s["q"][first + t, h].double() @ k[h // (Hq // Hkv)].T / math.sqrt(D)
                z = z.masked_fill(~seen, -math.inf)
                if s["sinks"] is not None:
                    z = torch.cat([z, s["sinks"][h].double().expand(len(t), 1)], 1)
                total = torch.logsumexp(z, 1)
                p = torch.exp(z - total[:, None])[:, :m]
                out[first + t, h] = p @ v[h // (Hq // Hkv)]
                lse[first + t, h] = total
        first += n
    return {"out": out, "lse": lse}
