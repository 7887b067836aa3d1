"""Differential attention in 64 bits, from its definition, with the bounds that the kernels' arithmetic allows."""
from __future__ import annotations

import math

import torch

from prompt_helpers import BF16_HALF, FP16_HALF, FP32_HALF, offsets, rows_of

D = 64  # elements of a head


class Maps:
    """y = A_0 V - lam A_1 V of every row, and mag, the same with magnitudes: sum A_0 |V| + |lam| sum A_1 |V|; none:
    rows that see no key; size: the largest scale * sum |q| |K|."""

    def __init__(self, rows, heads, device):
        self.y = torch.zeros((rows, heads, 2 * D), dtype=torch.float64, device=device)
        self.mag = torch.zeros_like(self.y)
        self.none = torch.ones(rows, dtype=torch.bool, device=device)
        self.size = 0.0


def maps_64(q, lens, pools, scales, keys, scale, lam, causal):
    """lens: rows of each sequence; keys: per sequence a list of (table row, tokens), one after the other (a shared
    prefix, then its own); lam [heads] or [rows, heads]."""
    hq, hkv = q.shape[1], pools[0].shape[2]
    g, heads, at = hq // hkv, hq // 2, offsets(lens)
    m = Maps(at[-1], heads, q.device)
    lam = lam.double().expand(at[-1], heads) if lam.dim() == 1 else lam.double()
    for b, n in enumerate(lens):
        c = sum(t for _, t in keys[b])
        if n == 0 or c == 0:
            continue
        k, v = (torch.cat([rows_of(x, scales, i, table, t) for table, t in keys[b]]) for i, x in enumerate(pools))
        rows = slice(at[b], at[b + 1])
        qq = q[rows].double().view(n, heads, 2, D)
        k = k.view(c, hkv // 2, 2, D).repeat_interleave(g, 1)  # [c, heads, map, D]
        v = v.view(c, hkv // 2, 2 * D).repeat_interleave(g, 1)
        lim = torch.full((n,), c, device=q.device)
        if causal:
            lim = (c - n + torch.arange(n, device=q.device) + 1).clamp(0, c)
        hidden = torch.arange(c, device=q.device)[None, :] >= lim[:, None]
        clean = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)
        wrong = (~torch.isfinite(v)).nonzero().tolist()
        m.none[rows] = lim == 0
        for t in range(2):
            s = torch.einsum("nhd,chd->hnc", qq[:, :, t], k[:, :, t]) * scale
            size = torch.einsum("nhd,chd->hnc", qq[:, :, t].abs(), k[:, :, t].abs()) * abs(scale)
            m.size = max(m.size, float(size.nan_to_num(0).max()))
            p = torch.softmax(s.masked_fill(hidden, -math.inf), -1).masked_fill((lim == 0)[:, None], 0)
            o = torch.einsum("hnc,chd->nhd", p, clean)
            for j, h, e in wrong:  # what a row does not see takes no part, whatever it holds
                o[lim > j, h, e] += v[j, h, e]
            f = 1.0 if t == 0 else lam[rows][..., None]
            m.y[rows] += o if t == 0 else -f * o
            m.mag[rows] += torch.einsum("hnc,chd->nhd", p, clean.abs()) * (1.0 if t == 0 else f.abs())
    return m


def finish_64(m, w, eps, out_scale):
    y = m.y
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
        y = torch.where(m.none[:, None, None], torch.zeros_like(y), y)
    return y * out_scale


def bounds(m, w, eps, out_scale, weight_half, e4m3, out_half):
    """How far an output may be from finish_64.

    Weights.  Scores: products summed in fp32, each addition off by at most 2^-23 of the sum of magnitudes (a step,
    for truncation), D of them and one for the scale: ds = (D + 1) 2^-23 size.  E4M3 pools: q's second term is off
    by 2^-18 of the row's largest where elements are below 2^-10 of it, at most that times sum |k| <= size *
    (largest / mean of |q|), taken as 64.  A weight is off by e^ds - 1, by 2^-21 for the exponential, and by its
    rounding, weight_half; a quotient of sums of such weights by twice the first two and once the last.  Sums over
    keys in fp32 add 2^-16 at these lengths, the difference and lam two roundings.  So y_i is off by
    e_i = rel mag_i.

    Norm.  With R = sqrt(mean y^2 + eps) and E = sqrt(mean e^2), the computed root is within E of R (a norm of
    (y, sqrt eps), triangle inequality), so y_i / R is off by at most e_i / (R - E) + |y_i| E / (R (R - E)); where
    E is not below R / 2 nothing is claimed.  mean, rsqrt, two products: 2^-19 of the result.  Then the rounding
    to the output's type."""
    ds = (D + 1) * 2.0 ** -23 * m.size + (2.0 ** -18 * m.size * 64 / 8 if e4m3 else 0.0)
    rel = 2 * (math.exp(ds) - 1 + 2.0 ** -21) + weight_half + 2.0 ** -16 + 2 * FP32_HALF
    e = rel * m.mag
    if w is None:
        off = e * abs(out_scale)
        size = m.y.abs() * abs(out_scale)
    else:
        r = (m.y.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        big = e.pow(2).mean(-1, keepdim=True).sqrt()
        ww = w.double().abs() * abs(out_scale)
        off = ww * (e / (r - big) + m.y.abs() * big / (r * (r - big)))
        off = torch.where(big < r / 2, off, math.inf)
        size = ww * m.y.abs() / r
    none = m.none[:, None, None]  # a row without keys is 0, not a result of these
    off, size = (torch.where(none, torch.zeros_like(x), x) for x in (off, size))
    off = off + 2.0 ** -19 * size
    return off + out_half * (size + off) + 1e-30


def halves(dtype):
    return FP32_HALF if dtype == torch.float32 else BF16_HALF


CHUNK_WEIGHT = {False: BF16_HALF, True: FP16_HALF}  # softmax weights of the chunk form, by pool type
STEP_WEIGHT = 2.0 ** -16  # of one token's forms: two 16-bit terms


def compare(got, ref, bound):
    got = got.double()
    same = torch.isnan(ref) & torch.isnan(got) | (torch.isinf(ref) & (got == ref))
    off = torch.where(same, 0.0, (got - ref).abs() - torch.where(torch.isfinite(ref), bound, 0.0))
    assert not torch.isnan(off).any(), "NaN where the definition has a value, or the reverse"
    if off.numel():
        assert float(off.max()) <= 0, (f"off by {float((got - ref).abs().nan_to_num(0).max()):.3e}, "
                                       f"{float(off.max()):.3e} past the bound")
