"""Rotary positions and the append to the paged cache, against their
definitions in 64 bits."""
import math

import numpy as np
import pytest

import attn_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _gen(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                        ("banded", dict(factor=8.0)),
                                        ("yarn", dict(factor=16.0, low=1.0, high=32.0, original_len=4096))])
def test_table(scaling, kw):
    """fp64 angles, one rounding to fp32; the scalings keep the fastest pair
    (all but "linear") and slow the slowest one by the factor."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    f, factor = ops.rope_frequencies(128, 500000.0, scaling, **kw)
    t = ops.rope_table(f, 301, factor, pos0=130000)
    a = torch.arange(130000, 130301, dtype=torch.float64)[:, None] * f
    want = torch.stack([a.cos(), a.sin()], -1) * factor
    assert (t.cpu().double() - want).abs().max() <= factor * 2.0 ** -24
    plain, _ = ops.rope_frequencies(128, 500000.0)
    if scaling != "linear":
        assert f[0] == plain[0]
    if kw:
        assert math.isclose(float(plain[-1] / f[-1]), kw["factor"], rel_tol=1e-12)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,H,D,rot,gap", [(1, 1, 128, 128, 0), (3, 72, 128, 128, 1024), (37, 5, 64, 64, 0),
                                           (19, 7, 128, 64, 24), (5, 3, 96, 32, 8), (4, 2, 80, 20, 0),
                                           (6, 3, 10, 6, 3), (9, 4, 64, 0, 0), (2, 130, 256, 256, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(dtype, T, H, D, rot, gap, interleaved):
    """Layouts, part of the head, odd head sizes, strided rows; forward,
    inverse, in place; the inverse is the gradient: <y, R x> = <R^T y, x>."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    dt = getattr(torch, dtype)
    rows = torch.randn((T, H * D + gap), generator=_gen(torch, T + D), device="cuda").to(dt)
    x = rows[:, :H * D].unflatten(1, (H, D))
    f, factor = ops.rope_frequencies(rot, 10000.0, "yarn", factor=4.0, high=32.0) if rot else (torch.empty(0), 1.0)
    table = ops.rope_table(f, 5000, factor) if rot else torch.empty((5000, 0, 2), device="cuda")
    pos = torch.randint(0, 5000, (T,), generator=_gen(torch, 1), device="cuda", dtype=torch.int32)
    pos[0] = 4999
    half = ref.BF16_HALF_ULP if dt == torch.bfloat16 else 0.0
    for inverse in (False, True):
        got = ops.rope(x, pos, table, interleaved=interleaved, inverse=inverse)
        want = ref.rotate(x.double(), pos, f.double(), factor, interleaved, inverse)
        tol = ref.rotate_bound(x.double(), pos, f.double(), factor, interleaved) + half * want.abs() * 1.01
        ref.assert_within(got, want, tol, f"rope inverse={inverse}")
        assert torch.equal(got[..., rot:], x[..., rot:])
    if dt == torch.float32 and rot:
        # the gradient against the formula's: the rotation is linear, so <g, R(x + d) - R(x)> is <R^T g, d>
        g = torch.randn((T, H, D), generator=_gen(torch, 3), device="cuda")
        back = ops.rope(g, pos, table, interleaved=interleaved, inverse=True).double()
        d = torch.randn((T, H, D), generator=_gen(torch, 4), device="cuda")
        xc = x.contiguous()
        moved = (ops.rope(xc + d, pos, table, interleaved=interleaved).double()
                 - ops.rope(xc, pos, table, interleaved=interleaved).double())
        lhs, rhs = (g.double() * moved).sum(), (back * ((xc + d).double() - xc.double())).sum()
        # each side: 4 half ulps per element of at most |g| (|x| + |d|) factor, twice
        scale = (g.abs().double() * (2 * xc.abs() + d.abs()).double()).sum() * 4 * factor
        assert abs(lhs - rhs) <= 8 * ref.F32_HALF_ULP * scale
    inplace = rows.clone()
    v = inplace[:, :H * D].unflatten(1, (H, D))
    ops.rope(v, pos, table, interleaved=interleaved, out=v)
    assert torch.equal(v, ops.rope(x, pos, table, interleaved=interleaved))
    assert torch.equal(inplace[:, H * D:], rows[:, H * D:])
    assert ops.device_error() == 0


def test_rope_position_outside_the_table():
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    f, factor = ops.rope_frequencies(64)
    table = ops.rope_table(f, 100, factor)
    x = torch.randn((4, 3, 64), device="cuda")
    pos = torch.tensor([0, 100, -1, 99], dtype=torch.int32, device="cuda")
    y = ops.rope(x, pos, table)
    assert ops.device_error() == 0x8
    assert torch.isnan(y[1:3]).all() and torch.isfinite(y[[0, 3]]).all()
    assert ops.device_error() == 0


# ------------------------------------------------------------------ append

LENS = {"one": ([1], [1]), "token": ([1, 1, 1, 1], [1, 700, 33, 4096]), "chunks": ([5, 0, 130, 1], [5, 9, 200, 65]),
        "many": ([1] * 40, list(range(1, 41)))}


def _append_case(torch, ops, fmt, dtype, D, Hq, Hkv, page, lens, rot, tokens_major=False, seed=0):
    n, m = LENS[lens]
    B, T = len(n), sum(n)
    counts = [-(-x // page) for x in m]
    P = sum(counts) + 2
    order = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).int()
    bt = torch.full((B, max(counts) + 1), -7, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        bt[b, :c] = order[at:at + c]
        at += c
    bt = bt.cuda()
    shape = (P, page, Hkv) if tokens_major else (P, Hkv, page)

    def new(last, dt):
        t = torch.zeros((*shape, last), dtype=dt, device="cuda")
        return t.transpose(1, 2) if tokens_major else t

    if fmt == "mxfp8":
        kv = ops.PagedKV(new(D, torch.uint8), new(D, torch.uint8), bt, new(D // 32, torch.uint8),
                         new(D // 32, torch.uint8))
    else:
        kv = ops.PagedKV(new(D, torch.bfloat16), new(D, torch.bfloat16), bt)
    rows = torch.randn((T, (Hq + 2 * Hkv) * D + 16), generator=_gen(torch, seed + 1), device="cuda")
    rows = rows.to(dtype)[:, :(Hq + 2 * Hkv) * D]
    qs = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    kl = torch.tensor(m, dtype=torch.int32, device="cuda")
    pos = torch.tensor([b - a + i for a, b in zip(n, m) for i in range(a)], device="cuda")
    seq = torch.tensor([b for b, a in enumerate(n) for _ in range(a)], device="cuda", dtype=torch.long)
    return kv, rows, qs, kl, pos, seq


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("D,Hq,Hkv,page,lens,rot,interleaved,tokens_major", [
    (128, 64, 8, 16, "token", 128, False, False), (128, 8, 1, 64, "chunks", 64, True, False),
    (64, 14, 2, 32, "many", 64, False, True), (96, 3, 3, 7, "chunks", 48, False, False),
    (32, 0, 2, 1, "token", 20, False, True), (256, 2, 1, 128, "one", 256, True, False),
    (64, 4, 4, 48, "chunks", 12, True, False), (128, 2, 2, 16, "many", 0, False, False)])
def test_append(fmt, dtype, D, Hq, Hkv, page, lens, rot, interleaved, tokens_major):
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    kv, rows, qs, kl, pos, seq = _append_case(torch, ops, fmt, getattr(torch, dtype), D, Hq, Hkv, page, lens, rot,
                                              tokens_major)
    f, factor = ops.rope_frequencies(rot, 10000.0, "yarn", factor=4.0, high=32.0) if rot else (torch.empty(0), 1.0)
    table = ops.rope_table(f, 4097, factor) if rot else None
    T = rows.shape[0]
    q = ops.kv_append(kv, rows, qs, kl, Hq, table, interleaved=interleaved)
    assert ops.device_error() == 0
    x = rows.double().view(T, -1, D)
    turned = ref.rotate(x[:, :Hq + Hkv], pos, f.double(), factor, interleaved)
    tol = ref.rotate_bound(x[:, :Hq + Hkv], pos, f.double(), factor, interleaved)
    ref.assert_within(q, turned[:, :Hq], tol[:, :Hq] + ref.BF16_HALF_ULP * turned[:, :Hq].abs() * 1.01, "q")
    at = kv.block_table[seq, pos // page].long()
    for name, want, t in (("k", turned[:, Hq:], tol[:, Hq:]), ("v", x[:, Hq + Hkv:], 0 * x[:, Hq + Hkv:])):
        cache = getattr(kv, name)
        got = cache[at, :, pos % page]
        rest = cache.clone()
        rest[at, :, pos % page] = 0
        assert not rest.any(), f"{name}: wrote elsewhere"
        if fmt == "bf16":
            ref.assert_within(got, want, t + ref.BF16_HALF_ULP * want.abs() * 1.01, name)
            continue
        scales = getattr(kv, name + "_scales")[at, :, pos % page]
        r, e = ref.mxfp8_quantize(want)
        same = scales.int() - 127 == e
        # a block whose maximum lies within fp32's error of a power of two may take the other exponent
        assert same.float().mean() > 0.999 and ((scales.int() - 127 - e).abs() <= 1).all()
        if name == "v":
            assert same.all()
            assert torch.equal(ref.e4m3_values("cuda")[got.long()], r)
        # a half step of E4M3 (2^-4 of the element, 2^-10 at the bottom), saturation up to 512 -> 448
        step = torch.exp2(e.double()).repeat_interleave(32, -1).view_as(want)
        v = ref.mxfp8_values(got, scales)
        top = (want.abs() / step).clamp(max=512)
        lim = torch.maximum(top * 2.0 ** -4, torch.full_like(top, 2.0 ** -10)) + (top - 448).clamp(min=0)
        ref.assert_within(v, want, 2 * lim * step + t, name)


def test_append_block_values():
    """MXFP8 blocks with zeros, subnormals, the top binade, infinities and NaN."""
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    D = 128
    rows = torch.zeros((1, 2 * D), device="cuda")
    v = rows[0, D:]
    v[0:32] = 0.0
    v[32:64] = torch.linspace(-511.9, 511.9, 32, device="cuda")
    v[64] = math.inf
    v[96:128] = 2.0 ** -140
    bt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    kv = ops.PagedKV.empty(1, 1, 16, D, bt, ops.KV_MXFP8)
    kv.k[:], kv.v[:] = 1, 1
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    ops.kv_append(kv, rows, one, one[1:], 0, None)
    r, e = ref.mxfp8_quantize(v.double()[None])
    assert torch.equal(kv.v_scales[0, 0, 0].int() - 127, e[0].int())
    assert torch.equal(ref.e4m3_values("cuda")[kv.v[0, 0, 0].long()], r[0])
    assert (kv.k[0, 0, 0] == 0).all() and (kv.k_scales[0, 0, 0] == 0).all()


def test_append_faults_and_rows_of_no_sequence():
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    D, page = 64, 16
    bt = torch.tensor([[0, 9], [1, -1]], dtype=torch.int32, device="cuda")
    kv = ops.PagedKV.empty(3, 1, page, D, bt)
    kv.k.zero_()
    f, factor = ops.rope_frequencies(D)
    table = ops.rope_table(f, 40, factor)
    rows = torch.randn((6, 3 * D), device="cuda")
    qs = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")

    def call(lens):
        q = torch.full((6, 1, D), 5.0, dtype=torch.bfloat16, device="cuda")
        ops.kv_append(kv, rows, qs, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1, table, q=q)
        return q, ops.device_error()

    q, err = call([2, 2])
    assert err == 0 and (q[4:] == 5).all() and torch.isfinite(q).all()
    q, err = call([17, 2])  # token 1 at position 16: page id 9 of 3
    assert err == 0x4 and torch.isnan(q[1]).all() and torch.isfinite(q[[0, 2, 3]]).all()
    q, err = call([2, 33])  # position 32: past the block table's row
    assert err == 0x4 and torch.isnan(q[3]).all()
    q, err = call([1, 2])   # two new tokens in a context of one
    assert err == 0x8 and torch.isnan(q[0]).all() and torch.isfinite(q[1]).all()
    q, err = call([2, 42])  # beyond the rotation table (and the block table)
    assert err == 0x8 and torch.isnan(q[2:4]).all()
    assert (kv.k[2] == 0).all()


THOUSANDS = [3900, 0, 1, 3] + [5 * i % 7 for i in range(230)] + [2099]
LENS["thousands"] = (THOUSANDS, [n + 13 * n % 50 for n in THOUSANDS])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("D,Hq,Hkv,interleaved", [(64, 1, 1, False), (64, 30, 5, True), (128, 26, 3, False)])
def test_append_more_tokens_than_blocks(fmt, dtype, D, Hq, Hkv, interleaved):
    """Blocks that take token after token, sequences of none to many tokens between them."""
    test_append(fmt, dtype, D, Hq, Hkv, 16, "thousands", D, interleaved, False)


def test_append_faults_among_many_tokens():
    torch = need_gpu()
    from gemm_decode_register_gb300 import ops

    D, page, n = 64, 16, 8000
    bt = torch.arange(n // page, dtype=torch.int32, device="cuda")[None].clone()
    bt[0, 300] = -1
    kv = ops.PagedKV.empty(n // page, 2, page, D, bt)
    kv.k.zero_()
    f, factor = ops.rope_frequencies(D)
    table = ops.rope_table(f, 7000, factor)
    rows = torch.randn((n + 5, 8 * D), device="cuda")
    qs, kl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n]))
    q = torch.full((n + 5, 4, D), 5.0, dtype=torch.bfloat16, device="cuda")
    ops.kv_append(kv, rows, qs, kl, 4, table, q=q)
    assert ops.device_error() == 0x4 | 0x8
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[300 * page:301 * page] = True
    bad[7000:] = True
    assert torch.equal(torch.isnan(q[:n]).all(2).all(1), bad) and torch.isfinite(q[:n][~bad]).all()
    assert (q[n:] == 5).all()
    stored = (kv.k != 0).any(3).any(1).view(-1)
    assert torch.equal(stored, ~bad)
