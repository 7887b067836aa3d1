"""The bounds of the differential attention's tests are tight: sums with a weight's second term left out, or with weights
kept without their factor, are outside them, and the arithmetic that the kernels state is inside."""
import pytest
import torch

from diff_tight import D, tight
from prompt_helpers import make_pool


def rounded(p, terms, kind, factor):
    """Weights as `terms` terms of 16 bits, times `factor` while they are rounded."""
    rest, total = p * factor, torch.zeros_like(p)
    for _ in range(terms):
        t = rest.to(kind).double()
        total, rest = total + t, rest - t
    return total / factor


def emulated(q, pools, scales, table, c, scale, lam, terms, kind, factor):
    """One sequence's outputs with rounded weights, everything else in 64 bits."""
    from prompt_helpers import rows_of

    hq, hkv = q.shape[1], pools[0].shape[2]
    g = hq // hkv
    k, v = (rows_of(x, scales, i, table, c) for i, x in enumerate(pools))
    k = k.view(c, hkv // 2, 2, D).repeat_interleave(g, 1)
    v = v.view(c, hkv // 2, 2 * D).repeat_interleave(g, 1)
    y = []
    for t in range(2):
        s = torch.einsum("hd,chd->hc", q[0].double().view(hq // 2, 2, D)[:, t], k[:, :, t]) * scale
        p = (s - s.amax(-1, keepdim=True)).exp()
        y.append(torch.einsum("hc,chd->hd", rounded(p, terms, kind, factor), v) / p.sum(-1)[:, None])
    return (y[0] - lam.double()[:, None] * y[1])[None]


def outside(e4m3, c, scale, terms, kind, factor, weights, ahead=None):
    k, v, scales, tables = make_pool([c], 4, D, e4m3, 21, device="cpu")
    g = torch.Generator().manual_seed(22)
    q = torch.randn((1, 8, D), generator=g).to(torch.bfloat16)
    lam = 0.4 + 0.3 * torch.randn(4, generator=g)
    if ahead is not None:
        q = torch.ones_like(q)
        kk = torch.zeros(k.shape)
        kk[..., 0] = torch.randint(-4, 5, kk.shape[:-1], generator=g) / 8.0
        kk[int(tables[0, 0]), 0] = ahead / 8
        v[int(tables[0, 0]), 0] = 0
        k = kk.to(k.dtype)
        if e4m3:
            scales = torch.stack((torch.ones_like(scales[0]), scales[1]))
    want, off = tight(q, [1], (k, v), scales, [[(tables[0], c)]], scale, lam, False, weights, c // 16 + 24)
    got = emulated(q, (k, v), scales, tables[0], c, scale, lam, terms, kind, factor)
    return float(((got - want).abs() / off).max())


@pytest.mark.parametrize("c", [2, 3, 5, 17])
def test_a_lost_second_term_shows(c):
    assert outside(True, c, 0.01, 2, torch.float16, 128.0, "fp16 pair") < 1
    assert outside(False, c, 0.01, 2, torch.bfloat16, 1.0, "bf16 pair") < 1
    assert outside(True, c, 0.01, 1, torch.float16, 128.0, "fp16 pair") > 1
    assert outside(False, c, 0.01, 1, torch.bfloat16, 1.0, "bf16 pair") > 1


def test_lost_small_weights_show():
    for terms, weights in ((2, "fp16 pair"), (1, "fp16")):
        assert outside(True, 512, 0.125, terms, torch.float16, 128.0, weights, ahead=18) < 1
        assert outside(True, 512, 0.125, terms, torch.float16, 1.0, weights, ahead=18) > 1
    assert outside(False, 512, 0.125, 2, torch.bfloat16, 1.0, "bf16 pair", ahead=18) < 1
