"""One token over an E4M3 pool, one key far ahead of all others and its value 0: the others' weights, below fp16's smallest
step of the largest, are all of the output."""
import pytest
import torch

from gpu_helpers import split_tokens
from prompt_helpers import FP32_HALF, make_pool, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("split", [None, 512, 64])
@pytest.mark.parametrize("ahead", [12, 20])
def test_one_key_far_ahead(pkv, ahead, split, hq, hkv, d):
    """Scores: products exact or off by 2^-23 of their sum of magnitudes, d + 4 times; exponentials and joins 2^-19; both in
    numerator and denominator.  Weights: two fp16 terms, 2^-22 of a weight or, times 2^15 relative to the maximum, half of
    fp16's smallest step, 2^-25, is 2^-40 of the largest.  Additions in fp32: two a block, and the joins."""
    ctx = [512, 700]
    k, v, scales, tables = make_pool(ctx, hkv, d, True, 3)
    g = torch.Generator().manual_seed(4)
    kk = torch.zeros(k.shape)
    kk[..., 0] = torch.randint(-4, 5, kk.shape[:-1], generator=g) / 8.0
    for b, at in enumerate((0, 600)):
        kk[int(tables[b, at // 16]), at % 16] = ahead / 8
        v.view(torch.uint8)[int(tables[b, at // 16]), at % 16] = 0
    k, scales = kk.to(k.dtype).cuda(), torch.stack((torch.ones_like(scales[0]), scales[1]))
    q = torch.ones((2, hq, d), dtype=torch.bfloat16, device="cuda")
    scale = 8.0 / d
    out = torch.empty((2, hq, d), device="cuda")
    with split_tokens(split):
        pkv.paged_decode_attention(q, k, v, tables, torch.tensor(ctx, dtype=torch.int32, device="cuda"), scale, out,
                                   scales=scales)
    assert pkv.check_device_status() == 0
    for b, c in enumerate(ctx):
        x, y = (rows_of(t, scales, i, tables[b], c).repeat_interleave(hq // hkv, 1) for i, t in enumerate((k, v)))
        s = torch.einsum("hd,chd->hc", q[b].double(), x) * scale
        size = torch.einsum("hd,chd->hc", q[b].double().abs(), x.abs()) * scale
        p = torch.softmax(s, -1)
        e = torch.expm1((d + 4) * 2.0 ** -23 * size + 2.0 ** -23 * size.amax(-1, keepdim=True)) + 2.0 ** -19
        want, mag = (torch.einsum("hc,chd->hd", p, w) for w in (y, y.abs()))
        off = torch.einsum("hc,chd->hd", p * (e + 2.0 ** -22) + 2.0 ** -40 * p.amax(-1, keepdim=True), y.abs())
        off = off + mag * ((p * e).sum(-1)[:, None] + (c // 8 + 32) * 2.0 ** -22 + 8 * FP32_HALF)
        assert bool(((out[b].double() - want).abs() <= 1.01 * off + FP32_HALF * want.abs()).all())
