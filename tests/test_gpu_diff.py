"""Differential attention over the paged cache against its definition in 64 bits: chunks, one token per sequence, and
shared prefixes; both pool types, query groups, lengths from none to long, split contexts, rows that see nothing,
pages holding NaN where nothing may be seen, and a run of the forms together as a server makes it."""
import math

import pytest
import torch

from diff_helpers import CHUNK_WEIGHT, STEP_WEIGHT, bounds, compare, finish_64, halves, maps_64
from gpu_helpers import split_tokens
from prompt_helpers import make_pool, offsets

pytestmark = pytest.mark.gpu

D = 64


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


class Job:
    """Inputs of a call: pool, queries, lam, norm weight."""

    def __init__(self, rows, ctx, hq, hkv, e4m3, seed, norm=True, per_token=False, extra=0, junk=math.nan, spread=1.0):
        self.k, self.v, self.scales, self.tables = make_pool(ctx, hkv, D, e4m3, seed, junk=junk)
        g = torch.Generator().manual_seed(seed + 1)
        self.q = (torch.randn((rows + extra, hq, D), generator=g) * spread).to(torch.bfloat16).cuda()
        lam = (rows + extra, hq // 2) if per_token else (hq // 2,)
        self.lam = (0.4 + 0.3 * torch.randn(lam, generator=g)).cuda()
        self.w = (1 + 0.2 * torch.randn(2 * D, generator=g)).to(torch.bfloat16).cuda() if norm else None
        self.e4m3, self.eps, self.out_scale = e4m3, 1e-5, 0.6 if norm else 1.0

    def keys(self):
        return dict(norm_weight=self.w, eps=self.eps, out_scale=self.out_scale, scales=self.scales)

    def row_lam(self, rows):
        return self.lam if self.lam.dim() == 1 else self.lam[:rows]


def check_chunk(pkv, lens, ctx, hq, hkv, e4m3, causal=True, seed=0, scale=0.125, split=None, extra=0, job=None,
                max_len=None, **kw):
    total = sum(lens)
    j = job or Job(total, ctx, hq, hkv, e4m3, seed, extra=extra, **kw)
    out = torch.full((total + extra, hq // 2, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.check_device_status()
    with split_tokens(split):
        pkv.paged_diff_prefill_attention(j.q, ints(offsets(lens)), j.k, j.v, j.tables, ints(ctx), scale, j.lam, out,
                                         causal=causal, max_context_len=max_len, **j.keys())
        flags = pkv.check_device_status()
    assert flags == 0, hex(flags)
    m = maps_64(j.q, lens, (j.k, j.v), j.scales, [[(j.tables[b], c)] for b, c in enumerate(ctx)], scale,
                j.row_lam(total), causal)
    compare(out[:total], finish_64(m, j.w, j.eps, j.out_scale),
            bounds(m, j.w, j.eps, j.out_scale, CHUNK_WEIGHT[e4m3], e4m3, halves(out.dtype)))
    assert not out[:total][m.none].any()
    assert bool((out[total:] == 7.0).all()), "rows behind the last sequence"
    return out


SHAPES = [(8, 8), (8, 4), (8, 2), (32, 4)]  # query groups 1, 2, 4, 8


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("lens,ctx", [
    ([1], [1]),
    ([1], [700]),
    ([5, 0, 1, 17], [5, 33, 129, 400]),
    ([300], [300]),
    ([129, 64, 511], [257, 64, 1300]),
])
def test_chunk(pkv, lens, ctx, hq, hkv, e4m3):
    check_chunk(pkv, lens, ctx, hq, hkv, e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", SHAPES)
def test_chunk_not_causal_without_norm_lam_per_token(pkv, hq, hkv, e4m3):
    check_chunk(pkv, [3, 40], [127, 1000], hq, hkv, e4m3, causal=False, norm=False, per_token=True)
    check_chunk(pkv, [200, 7, 333], [1500, 16, 128], hq, hkv, e4m3, causal=False, per_token=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [128, 256, 512])
@pytest.mark.parametrize("lens,ctx", [([2, 9], [1300, 700]), ([600, 31], [900, 31])])
def test_chunk_split_contexts(pkv, lens, ctx, split, e4m3):
    check_chunk(pkv, lens, ctx, 8, 2, e4m3, split=split)
    check_chunk(pkv, lens, ctx, 8, 4, e4m3, split=split, causal=False, norm=False, per_token=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [None, 128])
def test_chunk_rows_that_see_nothing(pkv, e4m3, split):
    check_chunk(pkv, [40, 300], [17, 100], 8, 2, e4m3, split=split)
    check_chunk(pkv, [4, 3], [0, 5], 8, 2, e4m3, split=split)
    check_chunk(pkv, [4, 300], [0, 0], 8, 2, e4m3, causal=False, split=split)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [None, 128])
def test_chunk_rows_without_keys_are_zero_at_eps_zero(pkv, e4m3, split):
    j = Job(40, [17], 8, 2, e4m3, 3)
    j.eps = 0.0
    check_chunk(pkv, [40], [17], 8, 2, e4m3, split=split, job=j)


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_rows_behind_the_last_sequence(pkv, e4m3):
    check_chunk(pkv, [33, 20], [50, 20], 8, 2, e4m3, extra=40)
    check_chunk(pkv, [33, 20], [500, 200], 8, 2, e4m3, extra=40, split=128)
    check_chunk(pkv, [0, 0], [50, 20], 8, 2, e4m3, extra=3, per_token=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
def test_chunk_scales(pkv, scale, e4m3):
    check_chunk(pkv, [70, 3], [400, 200], 8, 2, e4m3, scale=scale)


def grow(j, ctx):
    """Keys whose scores grow along the context."""
    for b, c in enumerate(ctx):
        for i in range((c + 15) // 16):
            f, blk = 0.02 * (1 + i), int(j.tables[b, i])
            if j.e4m3:
                j.k.view(torch.uint8)[blk] = (j.k[blk].float().nan_to_num(0) * f).clamp(-448, 448).to(
                    torch.float8_e4m3fn).view(torch.uint8)
            else:
                j.k[blk] = j.k[blk].float().nan_to_num(0) * f


@pytest.mark.parametrize("e4m3", [False, True])
def test_growing_scores_rescale(pkv, e4m3):
    ctx = [1500, 900]
    j = Job(302, ctx, 8, 2, e4m3, 5)
    grow(j, ctx)
    check_chunk(pkv, [300, 2], ctx, 8, 2, e4m3, scale=0.05, job=j)
    j = Job(2, ctx, 8, 2, e4m3, 6)
    grow(j, ctx)
    check_step(pkv, ctx, 8, 2, e4m3, scale=0.05, job=j)


@pytest.mark.parametrize("split", [None, 128])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_values_not_finite_reach_only_rows_that_see_them(pkv, e4m3, split, norm):
    lens, ctx = [200, 3], [330, 300]
    j = Job(203, ctx, 8, 4, e4m3, 9, norm=norm)
    for at, e, x in ((200, 3, math.nan), (317, 5, math.inf), (325, 5, -math.inf), (329, 60, math.nan)):
        blk = int(j.tables[0, at // 16])
        if e4m3:
            j.v.view(torch.uint8)[blk, at % 16, 1, e] = 0x7F
        else:
            j.v[blk, at % 16, 1, e] = x
    j.lam = j.lam.abs().neg()  # infinities of one sign add up
    check_chunk(pkv, lens, ctx, 8, 4, e4m3, split=split, job=j)


def test_chunk_strided_queries(pkv):
    lens, ctx = [70, 5], [100, 400]
    j = Job(75, ctx, 8, 2, False, 4)
    want = check_chunk(pkv, lens, ctx, 8, 2, False, job=j)
    packed = torch.randn((75, 12, D), device="cuda").to(torch.bfloat16)
    packed[:, :8] = j.q
    j.q = packed[:, :8]
    assert torch.equal(check_chunk(pkv, lens, ctx, 8, 2, False, job=j), want)


def test_chunk_long_context(pkv):
    check_chunk(pkv, [5], [70001], 8, 2, False, junk=None)
    check_chunk(pkv, [130], [66000], 4, 2, False, junk=None)


# ------------------------------------------------------------------ one token per sequence

def check_step(pkv, ctx, hq, hkv, e4m3, seed=0, scale=0.125, split=None, job=None, dtype=torch.float32, max_len=None, **kw):
    b = len(ctx)
    j = job or Job(b, ctx, hq, hkv, e4m3, seed, **kw)
    out = torch.full((b, hq // 2, 2 * D), 7.0, dtype=dtype, device="cuda")
    pkv.check_device_status()
    with split_tokens(split):
        pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, ints(ctx), scale, j.lam, out, max_context_len=max_len,
                                        **j.keys())
        flags = pkv.check_device_status()
    assert flags == 0, hex(flags)
    m = maps_64(j.q, [1] * b, (j.k, j.v), j.scales, [[(j.tables[i], c)] for i, c in enumerate(ctx)], scale, j.lam, False)
    compare(out, finish_64(m, j.w, j.eps, j.out_scale),
            bounds(m, j.w, j.eps, j.out_scale, STEP_WEIGHT, e4m3, halves(dtype)))
    assert not out[m.none].any()
    return out


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("ctx", [[1], [16], [777], [0, 5, 129, 2500, 16, 31]])
def test_step(pkv, ctx, hq, hkv, e4m3):
    check_step(pkv, ctx, hq, hkv, e4m3)
    check_step(pkv, ctx, hq, hkv, e4m3, dtype=torch.bfloat16, norm=False, per_token=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("split", [16, 48, 512])
def test_step_split_contexts(pkv, split, hq, hkv, e4m3):
    check_step(pkv, [0, 5, 129, 1500, 16, 31], hq, hkv, e4m3, split=split)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
def test_step_scales(pkv, scale, e4m3):
    check_step(pkv, [400, 3], 8, 2, e4m3, scale=scale)


@pytest.mark.parametrize("e4m3", [False, True])
def test_step_many_records(pkv, e4m3):
    check_step(pkv, [3000, 1100], 8, 2, e4m3, split=16)
    check_step(pkv, [100000], 4, 2, e4m3, junk=None)


# ------------------------------------------------------------------ shared prefixes

def check_shared(pkv, prefixes, members, tails, hq, hkv, e4m3, seed=0, scale=0.125, split=None, dtype=torch.float32,
                 job=None, max_members=None, **kw):
    """members: the sequences of each prefix."""
    b, P = len(tails), len(prefixes)
    j = job or Job(b, list(prefixes) + list(tails), hq, hkv, e4m3, seed, **kw)
    front = j.tables[:P, : max(1, max(prefixes) // 16)].contiguous()
    own = j.tables[P:].contiguous()
    prefix_of = [-1] * b
    for p, who in enumerate(members):
        for i in who:
            prefix_of[i] = p
    out = torch.full((b, hq // 2, 2 * D), 7.0, dtype=dtype, device="cuda")
    flat = [i for who in members for i in who]
    pkv.check_device_status()
    with split_tokens(split):
        pkv.cascade_diff_decode_attention(
            j.q, j.k, j.v, front, ints(prefixes), ints(offsets([len(w) for w in members])), ints(flat),
            ints(prefix_of), own, ints(tails), scale, j.lam, out,
            max_members=max(map(len, members)) if max_members is None else max_members, **j.keys())
        flags = pkv.check_device_status()
    assert flags == 0, hex(flags)
    keys = [([(front[prefix_of[i]], prefixes[prefix_of[i]])] if prefix_of[i] >= 0 else []) + [(own[i], t)]
            for i, t in enumerate(tails)]
    m = maps_64(j.q, [1] * b, (j.k, j.v), j.scales, keys, scale, j.lam, False)
    # a prefix's weights are two terms, but for E4M3 pools with a bf16 output: one, fp16
    weight = CHUNK_WEIGHT[True] if e4m3 and dtype == torch.bfloat16 else STEP_WEIGHT
    compare(out, finish_64(m, j.w, j.eps, j.out_scale), bounds(m, j.w, j.eps, j.out_scale, weight, e4m3, halves(dtype)))
    return out


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("prefixes,members,tails", [
    ([32], [[0]], [5]),
    ([16, 400], [[2, 0], [4]], [1, 16, 0, 7, 33]),
    ([2000, 0, 48], [[7, 1, 2], [3], [0, 5]], [0, 300, 1, 0, 700, 17, 16, 2]),
    ([656], [list(range(70))], [i % 40 for i in range(70)]),
])
def test_shared(pkv, prefixes, members, tails, hq, hkv, e4m3):
    check_shared(pkv, prefixes, members, tails, hq, hkv, e4m3)
    check_shared(pkv, prefixes, members, tails, hq, hkv, e4m3, norm=False, per_token=True, dtype=torch.bfloat16)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("split", [16, 48])
def test_shared_split_tails(pkv, split, e4m3):
    check_shared(pkv, [1600, 208], [[0, 3, 1], [4, 2]], [500, 30, 0, 129, 64, 700], 8, 2, e4m3, split=split)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
def test_shared_scales(pkv, scale, e4m3):
    check_shared(pkv, [320], [[0, 1, 2]], [40, 0, 9], 8, 2, e4m3, scale=scale)


def test_shared_without_members_is_the_decode(pkv):
    ctx = [40, 0, 200]
    j = Job(3, [16] + ctx, 8, 2, False, 2)
    own, c = j.tables[1:].contiguous(), ints(ctx)
    want = pkv.paged_diff_decode_attention(j.q, j.k, j.v, own, c, 0.125, j.lam, **j.keys())
    got = pkv.cascade_diff_decode_attention(j.q, j.k, j.v, j.tables[:1, :1].contiguous(), ints([16]), ints([0, 0]), ints([]),
                                            ints([-1, -1, -1]), own, c, 0.125, j.lam, max_members=0, **j.keys())
    assert torch.equal(got, want)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("e4m3", [False, True])
def test_a_served_layer(pkv, e4m3):
    """A prompt in two chunks (norm, rotation, append, attention), then decode steps of two samples that share its
    whole blocks, by the plain and by the cascade call."""
    hq, hkv, n = 16, 4, 75
    g = torch.Generator().manual_seed(11)
    blocks, step = 24, 3
    k = torch.zeros((blocks, 16, hkv, D), dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    scales = torch.full((2, hkv), 0.02, device="cuda") if e4m3 else None
    ids = torch.randperm(blocks, generator=g).to(torch.int32).cuda()
    prompt = ids[:5]  # 75 tokens: four whole blocks and 11 slots of a fifth
    freq, _ = pkv.rope_inv_freq(D, device="cuda")
    lam = pkv.diff_lambda(*(0.1 * torch.randn((hq // 2, D), generator=g) for _ in range(4)), 0.3).cuda()
    w = (1 + 0.1 * torch.randn(2 * D, generator=g)).to(torch.bfloat16).cuda()
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    keys = dict(norm_weight=w, out_scale=0.7, scales=scales)

    def append(tokens, positions, slots):
        x = torch.randn((tokens, hq + 2 * hkv, D), generator=g).to(torch.bfloat16).cuda()
        return pkv.qk_norm_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], ints(positions),
                                       torch.tensor(slots, device="cuda"), k, v, q_weight=wq, k_weight=wk,
                                       inv_freq=freq, scales=scales)

    def check(out, q, lens, key, causal, weight):
        m = maps_64(q, lens, (k, v), scales, key, 0.125, lam, causal)
        compare(out, finish_64(m, w, 1e-5, 0.7), bounds(m, w, 1e-5, 0.7, weight, e4m3, halves(out.dtype)))

    def slot(table, i):
        return int(table[i // 16]) * 16 + i % 16

    for lo, hi in ((0, 40), (40, n)):
        q = append(hi - lo, list(range(lo, hi)), [slot(prompt, i) for i in range(lo, hi)])
        out = pkv.paged_diff_prefill_attention(q, ints([0, hi - lo]), k, v, prompt[None].contiguous(), ints([hi]), 0.125, lam,
                                               **keys)
        check(out, q, [hi - lo], [[(prompt, hi)]], True, CHUNK_WEIGHT[e4m3])
    # two samples: the whole blocks shared, the fifth copied for the second
    pkv.copy_blocks(torch.tensor([[int(prompt[4]), int(ids[5])]], device="cuda"), k, v, scales)
    tails = torch.stack((torch.stack((prompt[4], ids[6])), torch.stack((ids[5], ids[7])))).contiguous()
    whole = torch.cat((prompt[:4].expand(2, 4), tails), 1).contiguous()
    for t in range(step + 3):
        at = n + t
        q = append(2, [at, at], [slot(whole[0], at), slot(whole[1], at)])
        c = ints([at + 1, at + 1])
        plain = pkv.paged_diff_decode_attention(q, k, v, whole, c, 0.125, lam, **keys)
        shared = pkv.cascade_diff_decode_attention(q, k, v, prompt[None, :4].contiguous(), ints([64]), ints([0, 2]),
                                                   ints([1, 0]), ints([0, 0]), tails, c - 64, 0.125, lam, max_members=2,
                                                   **keys)
        key = [[(whole[b], at + 1)] for b in range(2)]
        check(plain, q, [1, 1], key, False, STEP_WEIGHT)
        check(shared, q, [1, 1], key, False, CHUNK_WEIGHT[True] if e4m3 else STEP_WEIGHT)
    assert pkv.check_device_status() == 0


def test_lambda(pkv):
    g = torch.Generator().manual_seed(0)
    a, b, c, d = (0.2 * torch.randn((5, D), generator=g) for _ in range(4))
    got = pkv.diff_lambda(a, b, c, d, 0.35)
    want = [math.exp(float((a[i].double() * b[i].double()).sum())) - math.exp(float((c[i].double() * d[i].double()).sum()))
            + 0.35 for i in range(5)]
    assert got.dtype == torch.float32
    assert all(abs(float(x) - y) <= 2.0 ** -24 * abs(y) + 1e-15 for x, y in zip(got, want))
    assert pkv.diff_lambda(a[0], b[0], c[0], d[0], 0.35).shape == ()
