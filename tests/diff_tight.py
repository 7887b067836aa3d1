"""Differential attention without the norm in 64 bits, with a bound on each output element that is made key by key: tight
enough that a weight's second 16-bit term, or weights far below the largest, show when they are lost."""
from __future__ import annotations

import math

import torch

from prompt_helpers import BF16_HALF, FP16_HALF, FP32_HALF, offsets, rows_of

D = 64

# (relative, absolute in units of the row's largest weight) error of a softmax weight as the second product takes it:
# one or two 16-bit terms, each rounded to half a step of what is left.  fp16 weights carry a factor 2^7 relative to
# a reference that is at most the largest, so half of fp16's smallest step, 2^-25, is 2^-32 of it
WEIGHTS = {
    "bf16": (BF16_HALF, 0.0),
    "fp16": (FP16_HALF, 2.0 ** -32),
    "bf16 pair": (BF16_HALF ** 2, 0.0),
    "fp16 pair": (FP16_HALF ** 2, 2.0 ** -32),
}


def tight(q, lens, pools, scales, keys, scale, lam, causal, weights, adds, two_codes=False, out_half=FP32_HALF, out_scale=1.0):
    """(outputs [rows, heads, 2 D], bound on their error), out_scale (A_0 - lam A_1) V.  lens, keys as for maps_64.

    Scores.  (D + 4) roundings or truncations of 2^-23 of sum |q| |k| scale (products, the factor, the argument of the
    exponential), and one of the largest such sum for the reference: ds_j.  two_codes: q as two E4M3 terms, elements
    below 2^-9 of their row's largest off by 2^-17 of it; ds_j has scale 2^-17 largest sum |k| over those elements.
    A weight is off by d_j = e^ds_j - 1 + 2^-19 (exponentials: 2^-21 each, of the weight, of a moved reference and of the
    joins) in numerator and denominator alike, and in the numerator by its rounding (WEIGHTS).  adds additions in fp32
    of 2^-23 of the magnitudes' sum, in the numerator and in the denominator.  Quotient, V's scale, lam and the
    difference: eight roundings of 2^-24 of the magnitudes.  One per cent on top for products of errors.  Weights that
    are 0, of scores -inf, are exact."""
    rel, floor = WEIGHTS[weights]
    hq, hkv = q.shape[1], pools[0].shape[2]
    g, heads, at = hq // hkv, hq // 2, offsets(lens)
    y = torch.zeros((at[-1], heads, 2 * D), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(y)
    lam = lam.double().expand(at[-1], heads) if lam.dim() == 1 else lam.double()
    for b, n in enumerate(lens):
        c = sum(t for _, t in keys[b])
        if n == 0 or c == 0:
            continue
        k, v = (torch.cat([rows_of(x, scales, i, table, t) for table, t in keys[b] if t]) for i, x in enumerate(pools))
        rows = slice(at[b], at[b + 1])
        qq = q[rows].double().view(n, heads, 2, D)
        k = k.view(c, hkv // 2, 2, D).repeat_interleave(g, 1)
        v = v.view(c, hkv // 2, 2 * D).repeat_interleave(g, 1)
        lim = torch.full((n,), c, device=q.device)
        if causal:
            lim = (c - n + torch.arange(n, device=q.device) + 1).clamp(0, c)
        hidden = torch.arange(c, device=q.device)[None, :] >= lim[:, None]
        for t in range(2):
            x, kk = qq[:, :, t], k[:, :, t]
            s = (torch.einsum("nhd,chd->hnc", x, kk) * scale).masked_fill(hidden, -math.inf)
            p = torch.softmax(s, -1).masked_fill((lim == 0)[:, None], 0)
            size = torch.einsum("nhd,chd->hnc", x.abs(), kk.abs()) * abs(scale)
            size = torch.where(torch.isfinite(size) & ~hidden, size, 0)
            ds = (D + 4) * 2.0 ** -23 * size + 2.0 ** -23 * size.amax(-1, keepdim=True)
            if two_codes:
                top = x.abs().amax(-1, keepdim=True)
                low = torch.where(x.abs() < 2.0 ** -9 * top, 2.0 ** -17 * top, 0.0)
                ds = ds + torch.einsum("nhd,chd->hnc", low, kk.abs()) * abs(scale)
            d = torch.expm1(ds) + 2.0 ** -19
            o, mag = (torch.einsum("hnc,chd->nhd", p, w) for w in (v, v.abs()))
            e = torch.einsum("hnc,chd->nhd", p * (d + rel), v.abs())
            e = e + floor * torch.einsum("hnc,chd->nhd", p.amax(-1, keepdim=True) * (s > -math.inf), v.abs())
            e = e + mag * ((p * d).sum(-1).T[..., None] + 2 * adds * 2.0 ** -23 + 8 * 2.0 ** -24)
            f = 1.0 if t == 0 else lam[rows][..., None]
            y[rows] += o if t == 0 else -f * o
            bound[rows] += e if t == 0 else f.abs() * e
    y, bound = y * out_scale, bound * abs(out_scale) * 1.01
    return y, bound + out_half * (y.abs() + bound) + 1e-37
