"""Plain 64-bit definitions of the attention-side operators (rotary
positions, append to the paged cache, attention over it) on torch fp64
tensors, with the error bounds their tests use.  No code of the package."""
from __future__ import annotations

import math

import torch

BF16_HALF_ULP = 2.0 ** -8   # nearest-even to 8 significant bits (1 + 2^-8 lies half way between 1 and 1 + 2^-7)
F32_HALF_ULP = 2.0 ** -24


def rotate(x, pos, freq, factor, interleaved=False, inverse=False):
    """x fp64 [T][H][D]; pos [T]; freq fp64 [rot/2]."""
    rot = 2 * len(freq)
    a = pos.double()[:, None, None] * freq.to(x.device)
    c, s = torch.cos(a) * factor, torch.sin(a) * factor * (-1 if inverse else 1)
    y = x.clone()
    i = torch.arange(rot // 2, device=x.device)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., p] = x[..., p] * c - x[..., q] * s
    y[..., q] = x[..., q] * c + x[..., p] * s
    return y


def rotate_bound(x, pos, freq, factor, interleaved=False):
    """Largest error of the rotation in fp32: the table entries are rounded
    once, each product once and the sum once, so three half ulps of the two
    products' magnitudes; four cover the second-order terms."""
    rot = 2 * len(freq)
    b = torch.zeros_like(x)
    i = torch.arange(rot // 2, device=x.device)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    m = (x[..., p].abs() + x[..., q].abs()) * factor
    b[..., p] = m
    b[..., q] = m
    return 4 * F32_HALF_ULP * b


def mxfp8_quantize(x):
    """fp64 x [..., D] -> (elements, exponents e) with value element * 2^e per 32:
    e = floor(log2 max|x|) - 8, at least -127; nearest-even E4M3 with saturation.  A block with a NaN or an
    infinity gets e = 128 (the NaN scale) and zeros."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    fin = torch.isfinite(b).all(-1)
    _, ex = torch.frexp(torch.where(fin, amax, torch.ones_like(amax)))
    e = torch.where(amax == 0, torch.full_like(ex, -127), ex - 1 - 8).clamp(min=-127)
    v = torch.where(fin[..., None], b / torch.exp2(e.double())[..., None], torch.zeros_like(b))
    _, vx = torch.frexp(v)
    step = torch.exp2(torch.clamp(vx - 1, min=-6).double() - 3)  # spacing of E4M3 around v
    r = (v / step).round() * step
    r = r.clamp(-448, 448)
    return r.reshape(x.shape), torch.where(fin, e, torch.full_like(e, 128))


def e4m3_values(device):
    c = torch.arange(256, device=device)
    f, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(f == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(f.double() - 10))
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(c >= 128, -v, v)


def mxfp8_values(codes, scales):
    v = e4m3_values(codes.device)[codes.long()]
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return v * s.repeat_interleave(32, -1)


def seen(n, m, causal, window, device):
    """[n][m]: may new token i of n (position m - n + i) see key j?"""
    pos = m - n + torch.arange(n, device=device)[:, None]
    key = torch.arange(m, device=device)[None]
    ok = torch.ones((n, m), dtype=torch.bool, device=device)
    if causal:
        ok &= key <= pos
    if window:
        ok &= key > pos - window
    return ok


def attend(q, k, v, scale, causal=True, window=0, sinks=None):
    """q fp64 [n][Hq][D]; k, v fp64 [Hkv][m][D] (the context).  Returns out,
    lse and the largest errors of the kernels' arithmetic for each.

    Scores: fp32 sums of D exact products, each partial sum rounded or cut
    (2^-23 of the sum of magnitudes each): d <= (D + 4) 2^-23 |scale| sum|q k|.  Weights: off by the
    factor 1 + 2 d (both the score and the maximum) + 2^-19 for the power, and by a bf16 half ulp;
    the sum of the weights by 2 d + 2^-19 too.  So an output moves by at most
    (2^-8 + 4 d + 2^-18) sum p|v| / sum p, and its own rounding."""
    n, Hq, D = q.shape
    Hkv, m, _ = k.shape
    g = Hq // Hkv
    ok = seen(n, m, causal, window, q.device)
    out = torch.zeros((n, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for h in range(Hq):
        kh, vh = k[h // g], v[h // g]
        z = (q[:, h] @ torch.nan_to_num(kh).T) * scale  # non-finite keys are put back below
        bad = ~torch.isfinite(kh).all(1)
        if bad.any():
            z[:, bad] = torch.stack([(q[:, h] * kh[j]).sum(-1) for j in torch.nonzero(bad)[:, 0]], 1) * scale
        mag = (q[:, h].abs() @ torch.nan_to_num(kh).abs().T) * abs(scale)
        mag = torch.where(ok, mag, torch.zeros_like(mag)).amax(1) if m else torch.zeros(n, device=q.device).double()
        z = torch.where(ok, z, torch.full_like(z, -math.inf))
        top = z.amax(1) if m else torch.full((n,), -math.inf, device=q.device).double()
        if sinks is not None:
            top = torch.maximum(top, sinks[h].double())
        base = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p = torch.exp(z - base[:, None])
        p = torch.where(ok, p, torch.zeros_like(p))
        total = p.sum(1)
        if sinks is not None:
            total = total + torch.exp(sinks[h].double() - base)
        safe = torch.where(total == 0, torch.ones_like(total), total)
        # a key that a row may not see has no part in it, whatever its value
        acc = p @ torch.nan_to_num(vh, posinf=0.0, neginf=0.0)
        vbad = torch.nonzero(~torch.isfinite(vh).all(1))[:, 0].tolist()
        for j in vbad:
            rows = ok[:, j]
            acc[rows] = acc[rows] + p[rows, j, None] * torch.where(torch.isfinite(vh[j]), torch.zeros_like(vh[j]),
                                                                   vh[j])
        out[:, h] = acc / safe[:, None]
        lse[:, h] = torch.log(total) + base
        d = (D + 4) * 2.0 ** -23 * mag
        a = (p @ torch.nan_to_num(vh, nan=0.0, posinf=0.0, neginf=0.0).abs()) / safe[:, None]
        tol[:, h] = (BF16_HALF_ULP + 4 * d + 2.0 ** -18)[:, None] * a + BF16_HALF_ULP * out[:, h].abs() * 1.01 + 2.0 ** -134
        ltol[:, h] = 2 * d + 2.0 ** -18 * (1 + torch.nan_to_num(lse[:, h], neginf=0.0).abs())
    return out, lse, tol, ltol


def assert_within(got, want, tol, what):
    got, want = got.double(), want.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN positions differ"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fin = ~(nan | inf)
    assert torch.isfinite(got[fin]).all(), f"{what}: non-finite output"
    over = (got - want).abs()[fin] - tol.expand_as(want)[fin]
    if over.numel():
        assert over.max() <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} values off, worst by {float(over.max()):.3e}"
