"""Shared by the tests of the prompt side: pools with known contents and the operators'
definitions in 64 bits."""
from __future__ import annotations

import math

import torch

BLOCK = 16
BF16_HALF = 2.0 ** -8  # largest relative error of rounding to bf16
FP16_HALF = 2.0 ** -11
FP32_HALF = 2.0 ** -24
E4M3_HALF = 2.0 ** -4


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def make_pool(lens, hkv, d, e4m3, seed, device="cuda", spare=3, junk=None, spread=1.0):
    """Pools whose blocks are dealt out in a shuffled order; returns (k, v, scales, tables).  junk:
    a value written to every slot behind a sequence's last position and to the spare blocks."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
    blocks = sum(need) + spare
    ids = torch.randperm(blocks, generator=g)
    wide = max(1, max(need, default=1))
    tables = torch.full((len(lens), wide), blocks - 1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n].to(torch.int32)
        at += n
    k, v = (torch.randn((blocks, BLOCK, hkv, d), generator=g) * spread for _ in range(2))
    scales = None
    if e4m3:
        scales = torch.rand((2, hkv), generator=g) * 0.01 + 0.01
        k, v = ((x / scales[i][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn) for i, x in enumerate((k, v)))
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    if junk is not None:
        used = torch.zeros((blocks, BLOCK), dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(need[b]):
                used[tables[b, i], : min(BLOCK, n - i * BLOCK)] = True
        for x in (k, v):
            if e4m3:
                x.view(torch.uint8)[~used] = 0x7F  # NaN
            else:
                x[~used] = junk
    return (k.to(device), v.to(device), None if scales is None else scales.to(device), tables.to(device))


def rows_of(cache, scales, i, table, n):
    """The first n positions of a sequence in 64 bits: [n, hkv, d]."""
    x = cache[table[: (n + BLOCK - 1) // BLOCK].long()].double().flatten(0, 1)[:n]
    return x if scales is None else x * scales[i].double()[None, :, None]


def attention_64(q, lens, k, v, scales, tables, ctx, scale, causal):
    """Definition of the chunk attention; returns (out, lse, the same mean of |V|, and the largest
    scale * sum |q| |k|)."""
    hq, d = q.shape[1:]
    g = hq // k.shape[2]
    at = offsets(lens)
    out = torch.zeros((at[-1], hq, d), dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    lse = torch.full((at[-1], hq), -math.inf, dtype=torch.float64, device=q.device)
    size = 0.0
    for b, (n, c) in enumerate(zip(lens, ctx)):
        if n == 0 or c == 0:
            continue
        kk, vv = (rows_of(x, scales, i, tables[b], c) for i, x in enumerate((k, v)))
        qq = q[at[b]:at[b + 1]].double()
        kk, vv = kk.repeat_interleave(g, 1), vv.repeat_interleave(g, 1)
        s = torch.einsum("nhd,chd->hnc", qq, kk) * scale
        size = max(size, float((torch.einsum("nhd,chd->hnc", qq.abs(), kk.abs()) * abs(scale)).nan_to_num(0).max()))
        lim = torch.full((n,), c, device=q.device)
        if causal:
            lim = (c - n + torch.arange(n, device=q.device) + 1).clamp(0, c)
        hidden = torch.arange(c, device=q.device)[None, :] >= lim[:, None]
        s = s.masked_fill(hidden, -math.inf)
        lse[at[b]:at[b + 1]] = torch.logsumexp(s, -1).T
        p = torch.softmax(s, -1).masked_fill((lim == 0)[:, None], 0)
        # what a row does not see takes no part, whatever it holds
        clean = torch.nan_to_num(vv, nan=0.0, posinf=0.0, neginf=0.0)
        o = torch.einsum("hnc,chd->nhd", p, clean)
        wrong = ~torch.isfinite(vv)
        if bool(wrong.any()):
            for j, h, e in wrong.nonzero().tolist():
                o[lim > j, h, e] += vv[j, h, e]
        out[at[b]:at[b + 1]] = o
        mag[at[b]:at[b + 1]] = torch.einsum("hnc,chd->nhd", p, clean.abs())
    return out, lse, mag, size


def attention_bounds(out, mag, size, q, e4m3, d):
    """(bound on |out|, bound on |lse|) of the kernel's arithmetic.

    Scores: products summed in fp32, each addition off by at most 2^-23 of the sum of
    magnitudes (a step, for truncation), D of them and one for the scale: ds = (D + 1) 2^-23
    size.  E4M3 pools: q's second term is off by 2^-18 of the row's largest where elements are
    below 2^-10 of it, at most that times sum |k| <= size * (largest / mean of |q|), taken as 64.
    A weight is off by e^ds - 1, by 2^-21 for the exponential (approximate, argument rounded),
    and by its rounding to 16 bits; a quotient of sums of such weights by twice the first two
    and once the last.  The sums over keys in fp32 add 2^-16 at these lengths.  The result is
    rounded to bf16."""
    ds = (d + 1) * 2.0 ** -23 * size + (2.0 ** -18 * size * 64 / 8 if e4m3 else 0.0)
    half = FP16_HALF if e4m3 else BF16_HALF
    rel = 2 * (math.exp(ds) - 1 + 2.0 ** -21) + half + 2.0 ** -16
    bound = rel * mag + BF16_HALF * (out.abs() + rel * mag) + 1e-30
    return bound, ds + 2.0 ** -20 + 2.0 ** -16


def rope_64(x, w, eps, positions, inv_freq, interleaved, rope_scale):
    """Norm (w not None) and rotation of [T, H, D] in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    if inv_freq is None:
        return x
    half = inv_freq.shape[0]
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    t = (positions.double()[:, None] * inv_freq)[:, None]
    c, s = t.cos() * rope_scale, t.sin() * rope_scale
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y
