"""The blended frequencies against their definition, pair by pair, where the ramp ends inside the pairs and
where it runs past the last one."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


def yarn(rotary_dim, base, factor, original, fast=32.0, slow=1.0):
    """Pair i turns original * base^(-2i / R) / (2 pi) times over the original context; the index (not whole) that
    turns t times is where that equals t.  Kept up to the one for `fast` (rounded down, at least 0), divided by
    factor from the one for `slow` on (rounded up, at most R - 1), linear in the index between."""
    def index(t):
        return rotary_dim * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base))

    first, end = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rotary_dim - 1)
    out = []
    for i in range(rotary_dim // 2):
        f = base ** (-2 * i / rotary_dim)
        if end < 0 or i >= end and i > first:
            share = 1.0
        elif i <= first:
            share = 0.0
        else:
            share = (i - first) / (end - first)
        out.append(f * (1 - share) + f / factor * share)
    return torch.tensor(out, dtype=torch.float64)


@pytest.mark.parametrize("rotary_dim,base,factor,original", [
    (64, 1e4, 16.0, 4096), (128, 1e6, 4.0, 32768), (128, 5e5, 8.0, 8192),  # ends inside
    (128, 1e4, 4.0, 131072), (64, 1e4, 4.0, 65536), (32, 1e4, 4.0, 65536),  # every pair turns more than once
    (16, 100.0, 2.0, 1 << 20), (64, 1e4, 4.0, 1 << 30),  # the ramp starts behind the last pair: all kept
    (64, 1e4, 8.0, 150), (64, 1e4, 8.0, 2),  # it starts before the first; no pair turns once
])
def test_yarn_pair_by_pair(pkv, rotary_dim, base, factor, original):
    f, scale = pkv.rope_inv_freq(rotary_dim, base, scaling="yarn", factor=factor, original_max_position=original)
    assert math.isclose(scale, 0.1 * math.log(factor) + 1.0)
    # a power, a logarithm's quotient and a few products in fp64
    assert torch.allclose(f, yarn(rotary_dim, base, factor, original), rtol=1e-13)
