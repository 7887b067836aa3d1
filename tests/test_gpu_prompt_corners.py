"""Corners of the prompt side's calls that the tests by operator leave out."""
import math

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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def good_ranges(ip, rows):
    return [(b, ip[b], ip[b + 1]) for b in range(len(ip) - 1) if 0 <= ip[b] <= ip[b + 1] <= rows]


def test_workspace_without_memory_of_its_own(pkv):
    """The elements of an expanded or strided workspace are not the bytes behind it."""
    n, c, hq, hkv, d = 3, 900, 8, 2, 128
    k, v, _, tables = make_pool([c], hkv, d, False, 7)
    q = torch.randn((n, hq, d), device="cuda").to(torch.bfloat16)
    args = (q, ints([0, n]), k, v, tables, ints([c]), 0.1)
    with split_tokens(128):
        need = pkv.prefill_workspace_size(1, n, hq, hkv, d, tables.shape[1] * 16)
        assert need > 0
        want = pkv.paged_prefill_attention(*args)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        assert torch.equal(pkv.paged_prefill_attention(*args, workspace=ws), want)
        for bad in (ws[:1].expand(need), ws[:256].expand(need // 256 + 1, 256), torch.cat((ws, ws))[::2]):
            with pytest.raises(ValueError, match="contiguous"):
                pkv.paged_prefill_attention(*args, workspace=bad)
        ws.fill_(0xFF)
        assert torch.equal(pkv.paged_prefill_attention(*args, workspace=ws), want)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [None, 128])
@pytest.mark.parametrize("n,c,row", [(30, 12, 5), (40, 17, 5), (40, 17, 0), (300, 100, 195), (300, 300, None), (290, 200, 89)])
def test_queries_not_finite_of_rows_without_keys(pkv, n, c, row, split, e4m3):
    """A row at a negative position sees nothing: out 0 and lse -inf, whatever its query holds."""
    hq, hkv, d = 8, 2, 64
    k, v, scales, tables = make_pool([c], hkv, d, e4m3, 11, junk=float("nan"))
    g = torch.Generator().manual_seed(12)
    q = torch.randn((n, hq, d), generator=g).to(torch.bfloat16).cuda()
    for h, x in ((1, math.nan), (3, math.inf), (6, -math.inf)):
        q[n - 1, h, 7] = x
        if row is not None:
            q[row, h, 7] = x
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    with split_tokens(split):
        pkv.paged_prefill_attention(q, ints([0, n]), k, v, tables, ints([c]), 0.125, out, lse=lse, scales=scales)
    assert pkv.check_device_status() == 0
    blind = n - c
    assert bool((out[:blind] == 0).all()) and bool((lse[:blind] == -math.inf).all())
    bad = torch.isnan(out).any(-1)
    want = torch.zeros_like(bad)
    want[n - 1, [1, 3, 6]] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(lse), want)


@pytest.mark.parametrize("split", [None, 128])
@pytest.mark.parametrize("which", [0, 1])
def test_pool_scales_not_finite_and_rows_without_keys(pkv, which, split):
    n, c, hq, hkv, d = 300, 200, 8, 2, 64
    k, v, scales, tables = make_pool([c], hkv, d, True, 11)
    scales[which, 1] = math.nan
    g = torch.Generator().manual_seed(12)
    q = torch.randn((n, hq, d), generator=g).to(torch.bfloat16).cuda()
    lse = torch.full((n, hq), 7.0, device="cuda")
    with split_tokens(split):
        out = pkv.paged_prefill_attention(q, ints([0, n]), k, v, tables, ints([c]), 0.125, lse=lse, scales=scales)
    assert bool((out[:n - c] == 0).all()) and bool((lse[:n - c] == -math.inf).all())
    bad = torch.isnan(out)
    assert bool(bad[n - c:, 4:].all()) and not bool(bad[:, :4].any())


def good_ranges(ip, rows):
    return [(b, ip[b], ip[b + 1]) for b in range(len(ip) - 1) if 0 <= ip[b] <= ip[b + 1] <= rows]


# offsets of four ranges of 40 rows of which one entry or two are bad; no good range shares a row with another
DISORDER = [[0, 10, -5, 30, 40], [0, 10, 999, 30, 40], [0, -1, 12, 30, 40], [30, 40, 0, 10, 20], [5, 20, 3, 5, 5],
            [-2, 10, 24, 30, 50], [20, 40, 0, 20, 19]]


@pytest.mark.parametrize("ip", DISORDER, ids=str)
def test_gather_good_ranges_beside_bad_ones(pkv, ip):
    lens = [40, 40, 40, 40]
    k, v, _, tables = make_pool(lens, 2, 64, False, 3)
    ko, vo = (torch.full((40, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.check_device_status()
    pkv.paged_kv_gather(k, v, tables, ints(ip), ko, vo)
    assert pkv.check_device_status() == pkv.DEVFLAG_BAD_INDPTR
    for x, o in ((k, ko), (v, vo)):
        want = torch.full_like(o, 7.0)
        for b, first, last in good_ranges(ip, 40):
            want[first:last] = x[tables[b].long()].flatten(0, 1)[:last - first]
        assert torch.equal(o, want)


def test_gather_good_ranges_beside_bad_ones_of_many(pkv):
    """More ranges than a CTA keeps samples of."""
    n = 700
    k, v, _, tables = make_pool([3] * n, 1, 64, False, 5)
    ip = offsets([3] * n)
    for i, x in ((100, -5), (300, 1 << 20), (650, -1)):
        ip[i] = x
    rows = 3 * n
    ko, vo = (torch.full((rows, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.check_device_status()
    pkv.paged_kv_gather(k, v, tables, ints(ip), ko, vo)
    assert pkv.check_device_status() == pkv.DEVFLAG_BAD_INDPTR
    for x, o in ((k, ko), (v, vo)):
        want = torch.full_like(o, 7.0)
        for b, first, last in good_ranges(ip, rows):
            want[first:last] = x[tables[b].long()].flatten(0, 1)[:last - first]
        assert torch.equal(o, want)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [None, 128])
@pytest.mark.parametrize("times", [1, 8])  # 40 rows: a tile a work; 320: two
@pytest.mark.parametrize("ip", DISORDER, ids=str)
def test_attention_of_good_ranges_beside_bad_ones(pkv, ip, times, split, e4m3):
    hq, hkv, d, rows = 8, 2, 64, 40 * times
    ip = [x * times for x in ip]
    ctx = [700, 400, 330, 900]
    k, v, scales, tables = make_pool(ctx, hkv, d, e4m3, 6, junk=float("nan"))
    g = torch.Generator().manual_seed(4)
    q = torch.randn((rows, hq, d), generator=g).to(torch.bfloat16).cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    pkv.check_device_status()
    with split_tokens(split):
        pkv.paged_prefill_attention(q, ints(ip), k, v, tables, ints(ctx), 0.125, out, lse=lse, scales=scales)
    assert pkv.check_device_status() == pkv.DEVFLAG_BAD_INDPTR
    left = torch.ones(rows, dtype=torch.bool, device="cuda")
    for b, first, last in good_ranges(ip, rows):
        left[first:last] = False
        if first == last:
            continue
        qs = q[first:last]
        ref, ref_lse, mag, size = attention_64(qs, [last - first], k, v, scales, tables[b:b + 1], [ctx[b]], 0.125, True)
        bound, lse_bound = attention_bounds(ref, mag, size, qs, e4m3, d)
        assert bool(((out[first:last].double() - ref).abs() <= bound).all()), b
        assert bool(((lse[first:last].double() - ref_lse).abs() <= lse_bound + ref_lse.abs() * 2.0 ** -22).all()), b
    assert bool((out[left] == 7).all()) and bool((lse[left] == 7).all())


def test_split_attention_of_many_ranges_beside_bad_ones(pkv):
    """More ranges than a CTA of the merge has threads."""
    n, hq, hkv, d = 700, 4, 2, 64
    ctx = [150] * n
    k, v, _, tables = make_pool([150], hkv, d, False, 6)
    tables = tables.expand(n, -1).contiguous()
    ip = offsets([2] * n)
    for i, x in ((100, -5), (300, 1 << 20), (650, -1)):
        ip[i] = x
    g = torch.Generator().manual_seed(4)
    q = torch.randn((2 * n + 9, hq, d), generator=g).to(torch.bfloat16).cuda()
    for split in (None, 128):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pkv.check_device_status()
        with split_tokens(split):
            pkv.paged_prefill_attention(q, ints(ip), k, v, tables, ints(ctx), 0.125, out)
        assert pkv.check_device_status() == pkv.DEVFLAG_BAD_INDPTR
        left = torch.ones(len(q), dtype=torch.bool, device="cuda")
        for _, first, last in good_ranges(ip, len(q)):
            left[first:last] = False
        assert int(left.sum()) == 9 + 3 * 4 and bool((out[left] == 7).all())
        lens = [2] * n
        ref, _, mag, size = attention_64(q[:2 * n], lens, k, v, None, tables, ctx, 0.125, True)
        bound, _ = attention_bounds(ref, mag, size, q, False, d)
        off = (out[:2 * n].double() - ref).abs() - bound
        assert float(off[~left[:2 * n]].max()) <= 0


def test_tables_wider_than_any_context(pkv):
    """2^27 columns: columns times the block size passes 32 bits."""
    n, c, hq, hkv, d = 5, 300, 8, 2, 64
    k, v, _, tables = make_pool([c], hkv, d, False, 7)
    q = torch.randn((n, hq, d), device="cuda").to(torch.bfloat16)
    want = pkv.paged_prefill_attention(q, ints([0, n]), k, v, tables, ints([c]), 0.125, max_context_len=c)
    wide = torch.zeros((1, 1 << 27), dtype=torch.int32, device="cuda")
    wide[:, :tables.shape[1]] = tables
    pkv.check_device_status()
    got = pkv.paged_prefill_attention(q, ints([0, n]), k, v, wide, ints([c]), 0.125, max_context_len=c)
    assert pkv.check_device_status() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_frequencies_not_finite(pkv, bad, interleaved):
    """The pair of a frequency that is not finite has no angle: NaN, at position 0 too; the others are turned."""
    T, d, rot = 33, 64, 32
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((T, h, d), generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f, _ = pkv.rope_inv_freq(rot, device="cuda")
    kc, vc, _, _ = make_pool([T], 2, d, False, 1)
    slots = torch.arange(T, device="cuda")
    want = pkv.qk_norm_rope_append(q, k, v, pos, slots, kc, vc, inv_freq=f, interleaved=interleaved)
    k2, v2 = kc.clone(), vc.clone()
    f2 = f.clone()
    f2[5] = bad
    got = pkv.qk_norm_rope_append(q, k, v, pos, slots, k2, v2, inv_freq=f2, interleaved=interleaved)
    pair = [10, 11] if interleaved else [5, 21]
    rest = [i for i in range(d) if i not in pair]
    for a, b in ((got, want), (k2.view(-1, 2, d)[:T], kc.view(-1, 2, d)[:T])):
        assert bool(torch.isnan(a[..., pair]).all()) and torch.equal(a[..., rest], b[..., rest])


def test_small_elements_of_a_query_over_an_e4m3_pool(pkv):
    """Two E4M3 terms after the row's largest is taken into [128, 256): what is left after the first is held to
    half of E4M3's smallest step, 2^-10, so an element is exact from 2^-9 of the largest up and off by at most
    2^-17 of the largest below.  One key that meets only the small element; lse is its score."""
    d = 64
    k = torch.zeros((1, 16, 1, d), device="cuda")
    k[0, 0, 0, 1] = 448.0
    k = k.to(torch.float8_e4m3fn)
    scales = torch.tensor([[1.0], [1.0]], device="cuda")
    mant = 1 + torch.arange(128, device="cuda") / 128  # every bf16 of an octave
    for octave in range(0, 16):
        q = torch.zeros((128, 1, d), device="cuda")
        q[:, 0, 0] = 1.0
        q[:, 0, 1] = mant * 2.0 ** -octave / 2
        q = q.to(torch.bfloat16)
        lse = torch.empty((128, 1), device="cuda")
        pkv.paged_prefill_attention(q, ints([0, 128]), k, k, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                                    ints([1]), 1.0, causal=False, lse=lse, scales=scales)
        want = q[:, 0, 1].double() * 448
        # the two terms' products and their sum are exact; relative: log2(e) rounded, its product with the score,
        # two sums, ln 2 rounded and its product, below 8 roundings of 2^-24; absolute, at most 2^-19: the same two
        # sums with the weights' factor 2^7 (2^-21 of 7 together), log2 of it (two units in 7: 2^-20) and the
        # exponential (2^-22), times ln 2
        off = (lse[:, 0].double() - want).abs() - 8 * 2.0 ** -24 * want - 2.0 ** -19
        held = 0.0 if octave < 9 else 2.0 ** -17 * 448
        assert float(off.max()) <= held, octave
    assert pkv.check_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [None, 128])
@pytest.mark.parametrize("lens,ctx", [([3, 1, 8], [700, 300, 8]), ([300, 65, 700], [400, 65, 1500])])
def test_attention_in_place(pkv, lens, ctx, split, e4m3):
    hq, hkv, d = 16, 4, 128
    k, v, scales, tables = make_pool(ctx, hkv, d, e4m3, 7, junk=math.nan)
    q = torch.randn((sum(lens) + 5, hq, d), device="cuda").to(torch.bfloat16)
    rest = (k, v, tables, ints(ctx), 0.09)
    with split_tokens(split):
        want = pkv.paged_prefill_attention(q, ints(offsets(lens)), *rest, scales=scales)
        for _ in range(3):
            x = q.clone()
            got = pkv.paged_prefill_attention(x, ints(offsets(lens)), *rest, x, scales=scales)
            assert got is x and torch.equal(got[:-5], want[:-5]) and torch.equal(got[-5:], q[-5:])
        with pytest.raises(pkv.PkvError, match="overlaps"):
            pkv.paged_prefill_attention(q[:-1], ints(offsets(lens)), *rest, q[1:], scales=scales)
