"""Chunk attention over the paged cache against its definition in 64 bits: both pool types,
head dims and query groups, lengths from none to long, ragged and odd, causal and not, split
contexts, rows that see nothing, and pages holding NaN where nothing may be seen."""
import math
import os

import pytest
import torch

from gpu_helpers import split_tokens
from prompt_helpers import attention_64, attention_bounds, make_pool, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


def make(lens, ctx, hq, hkv, d, e4m3, seed, junk=float("nan"), extra=0, spread=1.0):
    k, v, scales, tables = make_pool(ctx, hkv, d, e4m3, seed, junk=junk)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn((sum(lens) + extra, hq, d), generator=g) * spread).to(torch.bfloat16).cuda()
    return q, k, v, scales, tables


def indptr(lens):
    return torch.tensor(offsets(lens), dtype=torch.int32, device="cuda")


def check(pkv, lens, ctx, hq, hkv, d, e4m3, causal=True, seed=0, scale=None, extra=0, split=None, spread=1.0, data=None,
          max_len=None):
    q, k, v, scales, tables = data or make(lens, ctx, hq, hkv, d, e4m3, seed, extra=extra, spread=spread)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    pkv.check_device_status()
    with split_tokens(split):
        pkv.paged_prefill_attention(q, indptr(lens), k, v, tables, c, scale, out, causal=causal, lse=lse,
                                    scales=scales, max_context_len=max_len)
        flags = pkv.check_device_status()
    assert flags == 0, hex(flags)
    total = sum(lens)
    ref, ref_lse, mag, size = attention_64(q[:total], lens, k, v, scales, tables, ctx, scale, causal)
    bound, lse_bound = attention_bounds(ref, mag, size, q, e4m3, d)
    got = out[:total].double()
    if total:
        both = torch.isnan(ref) & torch.isnan(got) | (torch.isinf(ref) & (got == ref))
        off = torch.where(both, 0.0, (got - ref).abs() - torch.where(torch.isfinite(ref), bound, 0.0))
        assert not torch.isnan(off).any(), "NaN where the definition has a value, or the reverse"
        assert float(off.max()) <= 0, f"off by {float((got - ref).abs().max()):.3e}, {float(off.max()):.3e} past the bound"
        empty = torch.isinf(ref_lse)
        assert torch.equal(torch.isinf(lse[:total]) & (lse[:total] < 0), empty)
        assert torch.equal(got[empty], torch.zeros_like(got[empty]))
        dl = (lse[:total].double() - ref_lse).abs()[~empty]
        far = float((dl - ref_lse[~empty].abs() * 2.0 ** -22).max()) if dl.numel() else 0.0
        assert far <= lse_bound, f"lse off by {far:.3e} of {lse_bound:.3e}"
    assert bool((out[total:] == 7.0).all()) and bool((lse[total:] == 7.0).all()), "rows behind the last sequence"
    return out


SHAPES = [(8, 8, 64), (8, 4, 128), (8, 2, 64), (16, 2, 128)]  # query groups 1, 2, 4, 8


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("lens,ctx", [
    ([1], [1]),
    ([1], [700]),
    ([5, 0, 1, 17], [5, 33, 129, 400]),
    ([300], [300]),
    ([129, 64, 511], [257, 64, 1300]),
])
def test_matches_definition(pkv, lens, ctx, hq, hkv, d, e4m3):
    check(pkv, lens, ctx, hq, hkv, d, e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("lens,ctx", [([3, 40], [127, 1000]), ([200, 7, 333], [1500, 16, 128])])
def test_not_causal(pkv, lens, ctx, hq, hkv, d, e4m3):
    check(pkv, lens, ctx, hq, hkv, d, e4m3, causal=False)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [128, 256, 512])
@pytest.mark.parametrize("lens,ctx", [([2, 9], [1300, 700]), ([600, 31], [900, 31])])
def test_split_contexts(pkv, lens, ctx, split, e4m3):
    check(pkv, lens, ctx, 8, 2, 128, e4m3, split=split)
    check(pkv, lens, ctx, 8, 2, 64, e4m3, split=split, causal=False)


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_that_see_nothing(pkv, e4m3):
    # more query rows than context: the first rows are at negative positions
    check(pkv, [40, 300], [17, 100], 8, 2, 128, e4m3)
    check(pkv, [40, 300], [17, 100], 8, 2, 128, e4m3, split=128)
    # contexts of length zero, causal and not
    check(pkv, [4, 3], [0, 5], 8, 2, 64, e4m3)
    check(pkv, [4, 300], [0, 0], 8, 2, 64, e4m3, causal=False)


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_behind_the_last_sequence(pkv, e4m3):
    check(pkv, [33, 20], [50, 20], 8, 2, 128, e4m3, extra=40)
    check(pkv, [33, 20], [500, 200], 8, 2, 128, e4m3, extra=40, split=128)
    check(pkv, [0, 0], [50, 20], 8, 2, 128, e4m3, extra=3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
def test_scales(pkv, scale, e4m3):
    check(pkv, [70, 3], [400, 200], 8, 2, 64, e4m3, scale=scale)


@pytest.mark.parametrize("e4m3", [False, True])
def test_growing_scores_rescale(pkv, e4m3):
    """Keys whose scores grow along the context: the reference moves step after step."""
    lens, ctx = [300, 2], [1500, 900]
    data = list(make(lens, ctx, 8, 2, 128, e4m3, 5))
    q, k, tables = data[0], data[1], data[4]
    for b, c in enumerate(ctx):
        for i in range((c + 15) // 16):
            f = 0.02 * (1 + i)
            blk = int(tables[b, i])
            if e4m3:
                k.view(torch.uint8)[blk] = (k[blk].float().nan_to_num(0) * f).clamp(-448, 448).to(
                    torch.float8_e4m3fn).view(torch.uint8)
            else:
                k[blk] = k[blk].float().nan_to_num(0) * f
    check(pkv, lens, ctx, 8, 2, 128, e4m3, data=data, scale=0.05)


@pytest.mark.parametrize("split", [None, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_values_not_finite_reach_only_rows_that_see_them(pkv, e4m3, split):
    lens, ctx = [200, 3], [330, 300]
    data = list(make(lens, ctx, 8, 2, 64, e4m3, 9))
    v, tables = data[2], data[4]
    for j, e, x in ((200, 3, math.nan), (317, 5, math.inf), (325, 5, -math.inf), (329, 60, math.nan)):
        blk = int(tables[0, j // 16])
        if e4m3:
            v.view(torch.uint8)[blk, j % 16, 1, e] = 0x7F
        else:
            v[blk, j % 16, 1, e] = x
    if e4m3:  # the only value that is not finite
        check(pkv, lens, ctx, 8, 2, 64, e4m3, data=data, split=split)
    else:
        check(pkv, lens, ctx, 8, 2, 64, e4m3, data=data, split=split)


def test_query_not_finite_stays_in_its_row(pkv):
    for e4m3 in (False, True):
        lens, ctx = [20], [150]
        data = list(make(lens, ctx, 8, 2, 64, e4m3, 11))
        data[0][4, 3, 7] = math.nan
        q = data[0]
        out = pkv.paged_prefill_attention(q, indptr(lens), data[1], data[2], data[4],
                                          torch.tensor(ctx, dtype=torch.int32, device="cuda"), 0.125, scales=data[3])
        bad = torch.isnan(out).all(-1)
        want = torch.zeros_like(bad)
        want[4, 3] = True
        assert torch.equal(bad, want) and torch.equal(torch.isnan(out).any(-1), want)


@pytest.mark.parametrize("e4m3", [False, True])
def test_small_queries_and_wide_ranges(pkv, e4m3):
    """Rows of q whose elements differ by many powers of two, and tiny rows."""
    lens, ctx = [64], [300]
    data = list(make(lens, ctx, 8, 2, 128, e4m3, 13))
    g = torch.Generator().manual_seed(3)
    e = torch.randint(-20, 1, (64, 8, 128), generator=g).cuda()
    data[0] = (data[0].float() * torch.pow(2.0, e.float())).to(torch.bfloat16)
    data[0][10] *= 2.0 ** -100
    data[0][11] = 0
    check(pkv, lens, ctx, 8, 2, 128, e4m3, data=data)


def test_long_context_long_offsets(pkv):
    """A pool of more than 2^31 elements (bf16): row offsets pass 32 bits."""
    hkv, d, blocks = 8, 128, (1 << 31) // (16 * 8 * 128) + 64
    k = torch.zeros((blocks, 16, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.arange(blocks - 40, blocks, dtype=torch.int32, device="cuda")
    k[-40:] = torch.randn((40, 16, hkv, d), generator=g, device="cuda", dtype=torch.bfloat16)
    v[-40:] = torch.randn((40, 16, hkv, d), generator=g, device="cuda", dtype=torch.bfloat16)
    q = torch.randn((9, 32, d), generator=g, device="cuda", dtype=torch.bfloat16)
    data = (q, k, v, None, ids[None].contiguous())
    check(pkv, [9], [637], 32, hkv, d, False, data=data)
    ko = torch.empty((640, hkv, d), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    pkv.paged_kv_gather(k, v, data[4], indptr([640]), ko, vo)
    assert torch.equal(ko, k[-40:].flatten(0, 1)) and torch.equal(vo, v[-40:].flatten(0, 1))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [None, 1 << 22])
@pytest.mark.parametrize("tokens", [10, 100])
def test_long_sums_keep_their_size(pkv, e4m3, split, tokens):
    """2^20 keys (256 blocks over and over) of values in [0.5, 1.5): all terms of the sums have one
    sign, and the tensor cores truncate their additions.  An accumulator takes at most 512 steps, 8 x 512
    additions, each off by at most 2^-23 of the sum: 2^-11.  Roundings of the weights and the output have
    either sign; over the 2,560 elements or more of the mean they leave under 2^-12.  One accumulator over all keys
    was off by 2^-7.2."""
    d, n = 64, 1 << 20
    g = torch.Generator().manual_seed(5)
    k = torch.randn((256, 16, 1, d), generator=g).to(torch.bfloat16).cuda()
    v = (torch.rand((256, 16, 1, d), generator=g) + 0.5).to(torch.bfloat16).cuda()
    scales = None
    if e4m3:
        k, v, scales = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), torch.ones(2, 1, device="cuda")
    q = torch.randn((tokens, 4, d), generator=g).to(torch.bfloat16).cuda()
    tables = (torch.arange(n // 16, dtype=torch.int32, device="cuda") % 256).view(1, -1)
    c = torch.tensor([n], dtype=torch.int32, device="cuda")
    with split_tokens(split):
        out = pkv.paged_prefill_attention(q, indptr([tokens]), k, v, tables, c, 0.125, causal=False, scales=scales)
        assert pkv.check_device_status() == 0
    s = torch.einsum("thd,jd->thj", q.double(), k.double().view(-1, d)) * 0.125
    ref = torch.softmax(s, -1) @ v.double().view(-1, d)
    off = (out.double() - ref) / ref
    assert abs(float(off.mean())) <= 2.0 ** -11 + 2.0 ** -12
    # one element: the output's rounding, the sums' 2^-11, and as much for the weights' (the mean of over a
    # thousand of their roundings)
    assert float(off.abs().max()) <= 2.0 ** -8 + 2.0 ** -10


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [None, 1 << 22])
@pytest.mark.parametrize("d", [64, 128])
def test_growing_scores_over_a_long_context(pkv, e4m3, split, d):
    """131,072 + 70,000 keys, the blocks of the later ones larger: references move after the outputs of
    the first 65,536 keys have been put aside, and the last part is cut inside a block.  The definition with
    every key counted as often as the tables have it."""
    n1, n2, tokens = 131072, 70003, 200
    g = torch.Generator().manual_seed(9)
    k = torch.randn((96, 16, 2, d), generator=g)
    k[32:64] *= 3.0
    k[64:] *= 9.0
    k = k.to(torch.bfloat16).cuda()
    v = torch.randn((96, 16, 2, d), generator=g).to(torch.bfloat16).cuda()
    scales = None
    if e4m3:
        scales = torch.tensor([[0.25, 0.5], [0.125, 0.0625]], device="cuda")
        k, v = ((x.float() / scales[i][:, None]).to(torch.float8_e4m3fn) for i, x in enumerate((k, v)))
    kf, vf = ((x.double() if scales is None else x.double() * scales[i].double()[:, None]) for i, x in enumerate((k, v)))
    q = torch.randn((tokens, 4, d), generator=g).to(torch.bfloat16).cuda()
    b = torch.arange((n1 + n2 + 15) // 16, dtype=torch.int32, device="cuda")
    tables = torch.where(b < 4096, b % 32, torch.where(b < n1 // 16, 32 + b % 32, 64 + b % 32)).to(torch.int32)
    c = torch.tensor([n1 + n2], dtype=torch.int32, device="cuda")
    lse = torch.empty((tokens, 4), device="cuda")
    with split_tokens(split):
        out = pkv.paged_prefill_attention(q, indptr([tokens]), k, v, tables.view(1, -1), c, 1 / math.sqrt(d),
                                          causal=False, lse=lse, scales=scales)
        assert pkv.check_device_status() == 0
    times = torch.zeros(96 * 16, dtype=torch.float64, device="cuda")
    at = tables.long().repeat_interleave(16) * 16 + torch.arange(16, device="cuda").repeat(len(tables))
    times.index_add_(0, at[:n1 + n2], torch.ones(n1 + n2, dtype=torch.float64, device="cuda"))
    for h in range(4):
        kh, vh = kf[:, :, h // 2].reshape(-1, d), vf[:, :, h // 2].reshape(-1, d)
        s = q[:, h].double() @ kh.T / math.sqrt(d) + torch.log(times)
        ref, ref_lse = torch.softmax(s, -1) @ vh, torch.logsumexp(s, -1)
        # a weight is off by at most 2^-8 of itself, the sums by 2^-11, so the output by that of the weighted
        # sizes, and half a step of its own; scores of up to 200 or so in fp32: 2^-24 x 2 x 200 x log2(e) in the weights
        size = torch.softmax(s, -1) @ vh.abs()
        bound = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13) * size + 2.0 ** -8 * ref.abs() + 1e-6
        assert bool(((out[:, h].double() - ref).abs() <= bound).all())
        assert float((lse[:, h].double() - ref_lse).abs().max()) <= 2.0 ** -10


def test_strided_queries(pkv):
    lens, ctx = [37, 90], [200, 90]
    q, k, v, scales, tables = make(lens, ctx, 8, 2, 128, False, 17)
    packed = torch.randn((127, 12, 128), device="cuda").to(torch.bfloat16)
    packed[:, :8] = q
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    a = pkv.paged_prefill_attention(q, indptr(lens), k, v, tables, c, 0.1)
    b = pkv.paged_prefill_attention(packed[:, :8], indptr(lens), k, v, tables, c, 0.1)
    assert torch.equal(a, b)


@pytest.mark.parametrize("split", [None, 256])
def test_repeats_bit_for_bit_and_is_independent_of_batch_order(pkv, split):
    lens, ctx = [100, 3, 260], [700, 513, 260]
    q, k, v, scales, tables = make(lens, ctx, 8, 2, 128, True, 21)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    with split_tokens(split):
        a = pkv.paged_prefill_attention(q, indptr(lens), k, v, tables, c, 0.1, scales=scales)
        b = pkv.paged_prefill_attention(q, indptr(lens), k, v, tables, c, 0.1, scales=scales)
        assert torch.equal(a, b)
        at = offsets(lens)
        order = [2, 0, 1]
        q2 = torch.cat([q[at[i]:at[i + 1]] for i in order])
        o2 = pkv.paged_prefill_attention(q2, indptr([lens[i] for i in order]), k, v, tables[order].contiguous(),
                                         c[order].contiguous(), 0.1, scales=scales)
    assert torch.equal(o2, torch.cat([a[at[i]:at[i + 1]] for i in order]))


def test_bad_data_is_flagged_and_not_followed(pkv):
    lens, ctx = [20, 30, 10], [100, 200, 60]
    q, k, v, scales, tables = make(lens, ctx, 8, 2, 64, False, 23, junk=0.0)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")

    def run(ip, t, cc):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pkv.check_device_status()
        pkv.paged_prefill_attention(q, ip, k, v, t, cc, 0.125, out)
        return out, pkv.check_device_status()

    good, flags = run(indptr(lens), tables, c)
    assert flags == 0
    t = tables.clone()
    t[1, 3] = k.shape[0]  # a block past the pool reads as zeros
    zero = make(lens, ctx, 8, 2, 64, False, 23, junk=0.0)
    zero[1][tables[1, 3]] = 0
    zero[2][tables[1, 3]] = 0
    out, flags = run(indptr(lens), t, c)
    assert flags == pkv.DEVFLAG_BAD_BLOCK_ID
    want = pkv.paged_prefill_attention(q, indptr(lens), zero[1], zero[2], tables, c, 0.125)
    assert torch.equal(out, want)
    c2 = c.clone()
    c2[2] = tables.shape[1] * 16 + 5  # clamped to the table
    _, flags = run(indptr(lens), tables.clone().clamp(min=0), c2)
    assert flags & pkv.DEVFLAG_BAD_CONTEXT_LEN
    ip = indptr(lens)
    ip[3] = 1000  # past the rows: that sequence is skipped
    out, flags = run(ip, tables, c)
    assert flags == pkv.DEVFLAG_BAD_INDPTR
    assert torch.equal(out[:50], good[:50]) and bool((out[50:] == 7).all())


def test_captured_graphs_share_no_workspace(pkv):
    """Two captured calls with split contexts, replayed beside each other on two streams."""
    jobs = []
    with split_tokens(128):
        for seed in (31, 32):
            lens, ctx = [3, 2], [1500, 1100]
            q, k, v, scales, tables = make(lens, ctx, 8, 2, 128, False, seed)
            c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
            ip = indptr(lens)
            want = pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.1)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.1)
            jobs.append((graph, out, want, torch.cuda.Stream(), (q, k, v, tables, c, ip)))
    for _ in range(20):
        for graph, _, _, s, _ in jobs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _, _ in jobs:
        assert torch.equal(out, want)


def test_other_stream(pkv):
    lens, ctx = [3, 2], [1500, 1100]
    q, k, v, scales, tables = make(lens, ctx, 8, 2, 128, True, 41)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    want = pkv.paged_prefill_attention(q, indptr(lens), k, v, tables, c, 0.1, scales=scales)
    ip = indptr(lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with split_tokens(256):
        got = [pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.1, scales=scales, stream=s) for _ in range(4)]
    s.synchronize()
    for o in got[1:]:
        assert torch.equal(o, got[0])
    assert float((got[0].float() - want.float()).abs().max()) < 0.05


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [None, 128])
def test_scores_not_finite(pkv, e4m3, split):
    """A key that is NaN spoils the rows that see it and no others, whichever part of the context it is in."""
    lens, ctx = [40, 2], [300, 260]
    for j in (3, 130, 280):
        data = list(make(lens, ctx, 8, 2, 64, e4m3, 61))
        k, tables = data[1], data[4]
        blk = int(tables[0, j // 16])
        if e4m3:
            k.view(torch.uint8)[blk, j % 16, 1, 9] = 0x7F
        else:
            k[blk, j % 16, 1, 9] = math.nan
        with split_tokens(split):
            out = pkv.paged_prefill_attention(data[0], indptr(lens), k, data[2], tables,
                                              torch.tensor(ctx, dtype=torch.int32, device="cuda"), 0.125, scales=data[3])
        bad = torch.isnan(out).all(-1)
        want = torch.zeros_like(bad)
        first = max(0, j - (300 - 40))
        want[first:40, 4:8] = True  # the rows at or past position j, the heads of kv head 1
        assert torch.equal(bad, want) and torch.equal(torch.isnan(out).any(-1), want)


@pytest.mark.parametrize("causal", [True, False])
def test_scales_of_the_pool_of_any_sign(pkv, causal):
    lens, ctx = [70, 300], [400, 500]
    data = list(make(lens, ctx, 8, 4, 64, True, 67))
    data[3][0, 1] *= -1
    data[3][0, 2] = 0
    data[3][1, 0] *= -1
    check(pkv, lens, ctx, 8, 4, 64, True, causal=causal, data=data)
    check(pkv, lens, ctx, 8, 4, 64, True, causal=causal, data=data, scale=-0.1, split=128)


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_sequences(pkv, e4m3):
    """More sequences than one warp looks over at a time, some without rows, some without context."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 4, (150,), generator=g).tolist()
    ctx = [max(n, int(c)) for n, c in zip(lens, torch.randint(0, 200, (150,), generator=g))]
    ctx[7] = 0
    check(pkv, lens, ctx, 8, 2, 64, e4m3)
    lens[100] = 900  # a long one among them: 256-row works on average no more
    ctx[100] = 1000
    check(pkv, lens, ctx, 8, 2, 64, e4m3)


@pytest.mark.parametrize("split", [None, 128])
def test_bad_range_leaves_its_rows(pkv, split):
    lens, ctx = [5, 6, 4], [300, 200, 260]
    q, k, v, scales, tables = make(lens, ctx, 8, 2, 64, False, 71, junk=0.0)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    ip = indptr(lens)
    ip[3] = 99
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.check_device_status()
    with split_tokens(split):
        pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.125, out)
    assert pkv.check_device_status() == pkv.DEVFLAG_BAD_INDPTR
    assert bool((out[11:] == 7).all()) and not bool((out[:11] == 7).all(-1).any())


def test_bad_range_behind_the_last_work_is_flagged(pkv):
    """64 sequences of a token fill every tile there can be; the 65th, whose range is bad, has none."""
    lens = [1] * 64
    q, k, v, scales, tables = make(lens, [20] * 64, 8, 2, 64, False, 72, junk=0.0)
    tables = torch.cat((tables, tables[:1]))
    c = torch.full((65,), 20, dtype=torch.int32, device="cuda")
    ip = torch.tensor(offsets(lens) + [70], dtype=torch.int32, device="cuda")
    pkv.check_device_status()
    out = pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.125)
    assert pkv.check_device_status() == pkv.DEVFLAG_BAD_INDPTR
    ip[65] = 64
    again = pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.125)
    assert pkv.check_device_status() == 0
    assert torch.equal(out, again)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(64, 8, 128), (40, 5, 64), (12, 3, 128)])
def test_many_short_works_with_one_tile(pkv, e4m3, hq, hkv, d):
    """Two-tile works whose second tile has no rows, hundreds of them: the softmax warps of that tile run
    ahead of the first tile's by as many works as they are told of.  (E4M3: they had counted as the
    first tile's, and scores were taken of the query rows of the work before.)"""
    for seed in range(8):
        g = torch.Generator().manual_seed(seed)
        group = hq // hkv
        lens = torch.randint(0, 320 // group, (40,), generator=g).tolist()
        ctx = [n + int(torch.randint(0, 3, (1,), generator=g)) for n in lens]
        q, k, v, scales, tables = make(lens, ctx, hq, hkv, d, e4m3, 100 + seed)
        c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        out = pkv.paged_prefill_attention(q, indptr(lens), k, v, tables, c, 1.0, scales=scales)
        assert pkv.check_device_status() == 0
        ref, _, mag, size = attention_64(q, lens, k, v, scales, tables, ctx, 1.0, True)
        bound, _ = attention_bounds(ref, mag, size, q, e4m3, d)
        # E4M3: weights are fp16 times 2^7 (2^15 at most), whose steps are 2^-24 at the least: a weight below
        # 2^-21 of the largest is off by up to 2^-32 of it, not of itself.  That shows where the larger weights
        # meet values that are 0; n keys of at most 448 times a scale add n 2^-32 448 times it
        small = max(ctx) * 2.0 ** -32 * 448 * float(scales[1].max()) if e4m3 else 0.0
        off = (out.double() - ref).abs() - bound - small
        assert not bool(torch.isnan(off).any()) and float(off.max()) <= 0, float(off.max())


def test_replay_with_other_lengths(pkv):
    """A captured call replayed after its offsets, lengths, tables and queries were overwritten: a padded batch
    whose real tokens change from step to step."""
    lens, ctx = [9, 30, 0, 25], [500, 30, 70, 400]
    q, k, v, scales, tables = make(lens, ctx, 8, 2, 128, False, 81)
    c, ip = torch.tensor(ctx, dtype=torch.int32, device="cuda"), indptr(lens)
    out = torch.empty_like(q)
    pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.1, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.1, out)
    for lens2, ctx2 in (([9, 30, 0, 25], [500, 30, 70, 400]), ([1, 1, 1, 1], [499, 30, 2, 17]), ([0, 0, 60, 2], [3, 3, 70, 390])):
        ip.copy_(indptr(lens2))
        c.copy_(torch.tensor(ctx2, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        want = torch.full_like(out, 7.0)
        pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.1, want)
        assert torch.equal(out, want) and bool((out[sum(lens2):] == 7).all())


def test_two_streams_at_once(pkv):
    jobs = []
    for seed in (91, 92):
        lens, ctx = [700, 3], [900, 2000]
        q, k, v, scales, tables = make(lens, ctx, 16, 2, 128, seed == 92, seed)
        c, ip = torch.tensor(ctx, dtype=torch.int32, device="cuda"), indptr(lens)
        want = pkv.paged_prefill_attention(q, ip, k, v, tables, c, 0.1, scales=scales)
        jobs.append(((q, ip, k, v, tables, c, 0.1), scales, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (args, scales, _, s) in enumerate(jobs):
            with torch.cuda.stream(s):
                got[i].append(pkv.paged_prefill_attention(*args, scales=scales))
    torch.cuda.synchronize()
    for i, (_, _, want, _) in enumerate(jobs):
        assert all(torch.equal(o, want) for o in got[i])


def test_binding_refusals_on_the_gpu(pkv):
    lens, ctx = [5], [40]
    q, k, v, scales, tables = make(lens, ctx, 8, 2, 64, False, 3)
    c, ip = torch.tensor(ctx, dtype=torch.int32, device="cuda"), indptr(lens)
    f = pkv.paged_prefill_attention
    with pytest.raises(TypeError):
        f(q.float(), ip, k, v, tables, c, 0.1)
    with pytest.raises(ValueError):
        f(q[:, :, :32], ip, k, v, tables, c, 0.1)
    with pytest.raises(ValueError):
        f(q, ip.cpu(), k, v, tables, c, 0.1)
    with pytest.raises(ValueError):
        f(q, ip.long(), k, v, tables, c, 0.1)
    with pytest.raises(TypeError):
        f(q, ip, k, v, tables.long(), c, 0.1)
    with pytest.raises(ValueError):
        f(q, ip, k, v[:, :, :1], tables, c, 0.1)
    with pytest.raises(ValueError):
        f(q, ip, k, v, tables, c, 0.1, torch.empty((5, 8, 64), device="cuda"))
    with pytest.raises(ValueError):
        f(q, ip, k, v, tables, c, 0.1, lse=torch.empty((5, 9), device="cuda"))
    with pytest.raises(pkv.PkvError):
        f(q, ip, k, v, tables, c, 0.1, max_context_len=10 ** 6)
    with pytest.raises(pkv.PkvError):
        f(q[:, :6].contiguous(), ip, k, v, tables, c, 0.1)
    with pytest.raises(ValueError):
        f(q, ip, k, v, tables, c, 0.1, scales=torch.ones((2, 3), device="cuda"))
    with split_tokens(128):  # a workspace that is too small
        q2, k2, v2, _, t2 = make([5], [400], 8, 2, 64, False, 3)
        c2 = torch.tensor([400], dtype=torch.int32, device="cuda")
        with pytest.raises(pkv.PkvError) as e:
            f(q2, ip, k2, v2, t2, c2, 0.1, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
        assert e.value.status == pkv.PKV_ERR_WORKSPACE
    with pytest.raises(ValueError):
        pkv.qk_norm_rope_append(q, q[:, :2], q[:, :2], None, torch.arange(5, device="cuda"), k, v,
                                inv_freq=torch.ones(32, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        pkv.paged_kv_gather(k, v, tables, ip, q[:, :3], q[:, :3])
