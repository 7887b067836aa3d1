"""Differential attention where its numbers are hard to hold, against 64 bits, with bounds made key by key: weights far
below the largest, weights in two 16-bit terms, keys and values that are not finite, long runs of a shared prefix."""
import math

import pytest
import torch

from diff_helpers import compare
from diff_tight import tight
from gpu_helpers import split_tokens
from prompt_helpers import BF16_HALF, FP32_HALF, offsets
from test_gpu_diff import D, SHAPES, Job, grow, ints
from test_gpu_wait_timeout import env

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


def halves(dtype):
    return FP32_HALF if dtype == torch.float32 else BF16_HALF


def step(pkv, j, ctx, scale=0.125, split=None, dtype=torch.float32):
    """One token a sequence, checked.  Additions to a warp's accumulator: two a block of a run, of which it has half at
    most; then the joins of warps and runs."""
    out = torch.full((len(ctx), j.q.shape[1] // 2, 2 * D), 7.0, dtype=dtype, device="cuda")
    with split_tokens(split):
        pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, ints(ctx), scale, j.lam, out, **j.keys())
    assert pkv.check_device_status() == 0
    run = min(max(ctx), split or 512) // 16
    want, off = tight(j.q, [1] * len(ctx), (j.k, j.v), j.scales, [[(j.tables[i], c)] for i, c in enumerate(ctx)], scale, j.lam,
                      False, "fp16 pair" if j.e4m3 else "bf16 pair", 2 * (run + 4) + 16 + max(ctx) // 64, out_half=halves(dtype))
    compare(out, want, off)
    return out


def chunk(pkv, j, lens, ctx, scale=0.125, split=None, causal=True):
    out = torch.full((sum(lens), j.q.shape[1] // 2, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    with split_tokens(split):
        pkv.paged_diff_prefill_attention(j.q, ints(offsets(lens)), j.k, j.v, j.tables, ints(ctx), scale, j.lam, out,
                                         causal=causal, **j.keys())
    assert pkv.check_device_status() == 0
    want, off = tight(j.q, lens, (j.k, j.v), j.scales, [[(j.tables[i], c)] for i, c in enumerate(ctx)], scale, j.lam, causal,
                      "fp16" if j.e4m3 else "bf16", 8 * (max(ctx) // 128 + 2) + 64, j.e4m3, BF16_HALF)
    compare(out, want, off)
    return out


def shared(pkv, j, prefixes, members, tails, scale=0.125, dtype=torch.float32, run=None):
    """run: blocks of a run of the prefix pass (a step, 128 keys, is 16 additions to an accumulator where weights have two
    terms, else 8)."""
    n, P = len(tails), len(prefixes)
    front, own = j.tables[:P, : max(1, max(prefixes) // 16)].contiguous(), j.tables[P:].contiguous()
    of = [-1] * n
    for p, who in enumerate(members):
        for i in who:
            of[i] = p
    out = torch.full((n, j.q.shape[1] // 2, 2 * D), 7.0, dtype=dtype, device="cuda")
    with env(**({} if run is None else {"PKV_PREFIX_SPLIT_BLOCKS": str(run)})):
        pkv.cascade_diff_decode_attention(
            j.q, j.k, j.v, front, ints(prefixes), ints(offsets([len(w) for w in members])),
            ints([i for who in members for i in who]), ints(of), own, ints(tails), scale, j.lam, out,
            max_members=max(map(len, members)), **j.keys())
    assert pkv.check_device_status() == 0
    keys = [([(front[of[i]], prefixes[of[i]])] if of[i] >= 0 else []) + [(own[i], t)] for i, t in enumerate(tails)]
    one = j.e4m3 and dtype == torch.bfloat16
    steps = min(64, max(prefixes) // 128 + 1)
    want, off = tight(j.q, [1] * n, (j.k, j.v), j.scales, keys, scale, j.lam, False,
                      "fp16" if one else "fp16 pair" if j.e4m3 else "bf16 pair", (8 if one else 16) * steps + 128, j.e4m3,
                      halves(dtype))
    compare(out, want, off)
    return out


# ------------------------------------------------------------------ weights far below the largest

def sink(j, where, ahead):
    """The key at each (sequence, position) ahead of all others by `ahead` in both maps, its value 0; the others' scores
    are small and their values ordinary."""
    g = torch.Generator().manual_seed(17)
    j.q = torch.ones_like(j.q)
    k = torch.zeros(j.k.shape)
    k[..., 0] = torch.randint(-4, 5, j.k.shape[:-1], generator=g) / 8.0
    for b, at in where:
        k[int(j.tables[b, at // 16]), at % 16] = ahead / 8  # (64 elements, scale 1/8)
        j.v[int(j.tables[b, at // 16]), at % 16] = 0
    j.k = k.to(j.k.dtype).cuda()
    if j.e4m3:
        j.scales = torch.stack((torch.ones_like(j.scales[0]), j.scales[1]))


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("split", [None, 512])
@pytest.mark.parametrize("ahead", [12, 18])
@pytest.mark.parametrize("e4m3", [False, True])
def test_step_one_key_far_ahead(pkv, e4m3, ahead, split, hq, hkv):
    """Ahead by 18 (2^26), the others' weights are below fp16's smallest step, and all of the output."""
    ctx = [512, 700]
    j = Job(2, ctx, hq, hkv, e4m3, 3, norm=False, junk=None)
    sink(j, [(0, 0), (1, 600)], ahead)
    step(pkv, j, ctx, split=split)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_one_key_far_ahead(pkv, e4m3, dtype):
    prefixes, members, tails = [512, 256], [[0, 2], [1]], [300, 0, 40, 513]
    j = Job(4, prefixes + tails, 8, 2, e4m3, 5, norm=False, junk=None)
    sink(j, [(0, 3), (1, 255), (5, 100)], 18)
    shared(pkv, j, prefixes, members, tails, dtype=dtype, run=1000)


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_one_key_far_ahead(pkv, e4m3):
    lens, ctx = [40, 3], [512, 300]
    j = Job(43, ctx, 8, 2, e4m3, 6, norm=False, junk=None)
    sink(j, [(0, 0), (1, 130)], 18)
    chunk(pkv, j, lens, ctx)


# ------------------------------------------------------------------ keys that are infinite

def infinite(j, maps, keys):
    """Scores of -inf under the maps at `keys` of the first sequence: one element of the keys of every pair -inf, of
    every query positive."""
    for t in maps:
        j.q[:, t::2, 5] = j.q[:, t::2, 5].abs() + 0.5
        for at in keys:
            j.k[int(j.tables[0, at // 16]), at % 16, t::2, 5] = -math.inf


MAPS = [(0,), (1,), (0, 1)]
INFINITE = [range(0, 1), range(77, 78), range(0, 200), range(150, 160), range(0, 300)]


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("split", [None, 16, 512])
@pytest.mark.parametrize("maps", MAPS)
@pytest.mark.parametrize("keys", INFINITE, ids=str)
def test_step_infinite_keys(pkv, keys, maps, split, hq, hkv):
    """Keys whose score is -inf under one map have weight 0 there, the first ones of a warp too, and theirs under the other;
    a row of nothing but such scores has no value."""
    ctx = [300, 40]
    j = Job(2, ctx, hq, hkv, False, 4, norm=False)
    infinite(j, maps, keys)
    out = step(pkv, j, ctx, split=split)
    assert bool(out[0].isnan().all()) == (len(keys) == 300) and not out[1].isnan().any()


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("split", [None, 128])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("maps", MAPS)
@pytest.mark.parametrize("keys", INFINITE, ids=str)
def test_chunk_infinite_keys(pkv, keys, maps, norm, split, hq, hkv):
    """(A row sees some of the keys: only the ones that see no other have no value.)"""
    lens, ctx = [290, 3], [300, 40]
    j = Job(293, ctx, hq, hkv, False, 4, norm=False)
    infinite(j, maps, keys)
    out = chunk(pkv, j, lens, ctx, split=split)
    if norm:  # NaN where there is none without it, in the whole row
        j.w = torch.ones(2 * D, dtype=torch.bfloat16, device="cuda")
        with split_tokens(split):
            got = pkv.paged_diff_prefill_attention(j.q, ints(offsets(lens)), j.k, j.v, j.tables, ints(ctx), 0.125, j.lam,
                                                   **j.keys())
        assert torch.equal(got.isnan(), out.isnan())


@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("maps", MAPS)
@pytest.mark.parametrize("keys", [range(0, 1), range(0, 200), range(0, 256)], ids=str)
def test_shared_infinite_keys(pkv, keys, maps, hq, hkv):
    """In a prefix; a member without other keys sees nothing else, one with some does."""
    prefixes, members, tails = [256, 16], [[0, 2], [1]], [300, 9, 0, 64, 0]
    j = Job(5, prefixes + tails, hq, hkv, False, 7, norm=False)
    infinite(j, maps, keys)
    out = shared(pkv, j, prefixes, members, tails)
    assert bool(out[2].isnan().all()) == (len(keys) == 256) and not out[[0, 1, 3, 4]].isnan().any()
    assert not out[4].any()


# ------------------------------------------------------------------ two terms

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", SHAPES)
def test_weights_in_two_terms(pkv, hq, hkv, e4m3):
    """Few keys and small scores: an fp32 output shows each weight's bits."""
    ctx = [2, 3, 5, 4, 17]
    step(pkv, Job(5, ctx, hq, hkv, e4m3, 8, norm=False), ctx, scale=0.01)
    j = Job(3, [16, 32, 3, 0, 2], hq, hkv, e4m3, 9, norm=False)
    shared(pkv, j, [16, 32], [[0, 1], [2]], [3, 0, 2], scale=0.01)


# ------------------------------------------------------------------ long runs of a prefix

@pytest.mark.parametrize("run", [None, 8, 40, 128, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 2), (16, 2)])
def test_shared_long_runs(pkv, hq, hkv, e4m3, dtype, run):
    """Runs of 1, 5, 16 and, at 8192 tokens, as many steps as a run may have."""
    prefixes, members, tails = [2000, 8192, 336], [[4, 0], [2, 5, 3], [6]], [5, 300, 0, 17, 64, 1, 700]
    j = Job(7, prefixes + tails, hq, hkv, e4m3, 11, norm=False, per_token=True)
    shared(pkv, j, prefixes, members, tails, dtype=dtype, run=run)


@pytest.mark.parametrize("run", [None, 1000])
@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_values_of_one_sign(pkv, e4m3, run):
    """Where truncated sums are all off to the same side."""
    prefixes, members, tails = [8192], [[0, 1]], [0, 40]
    j = Job(2, prefixes + tails, 8, 2, e4m3, 12, norm=False)
    if e4m3:
        j.v = (j.v.view(torch.uint8) & 0x7F).view(torch.float8_e4m3fn)
    else:
        j.v = j.v.abs()
    j.lam = -j.lam.abs()
    shared(pkv, j, prefixes, members, tails, scale=0.01, run=run)


@pytest.mark.parametrize("run", [None, 40, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_growing_scores(pkv, e4m3, dtype, run):
    """The reference moves again and again, and the outputs are rescaled."""
    prefixes, tails = [2000], [30, 0, 1]
    j = Job(3, prefixes + tails, 8, 2, e4m3, 13, norm=False)
    grow(j, prefixes + tails)
    shared(pkv, j, prefixes, [[0, 2]], tails, scale=0.05, dtype=dtype, run=run)


# ------------------------------------------------------------------ values that are not finite

@pytest.mark.parametrize("hq,hkv", SHAPES)
@pytest.mark.parametrize("kind,e4m3", [("nan", False), ("inf", False), ("nan", True)])  # (E4M3 has no infinity)
def test_one_token_values_not_finite(pkv, kind, e4m3, hq, hkv):
    """A value inside a context that is not finite makes its own element, of its own kv pair's heads, of the sequences
    that see it, infinite or NaN (with the norm their whole rows), and nothing else."""

    def spoil(j, row, at, head, e):
        blk = int(j.tables[row, at // 16])
        if e4m3:
            j.v.view(torch.uint8)[blk, at % 16, head, e] = 0x7F
        else:
            j.v[blk, at % 16, head, e] = math.nan if kind == "nan" else math.inf

    head = hkv - 1  # the last pair's second half
    heads = slice(hq // 2 - hq // hkv, hq // 2)
    touched = torch.zeros((4, hq // 2, 2 * D), dtype=torch.bool, device="cuda")
    touched[1, heads, D + 9] = True
    ctx = [40, 300, 17, 0]
    for norm in (False, True):
        j = Job(4, ctx, hq, hkv, e4m3, 14, norm=norm)

        def run():
            return pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, ints(ctx), 0.125, j.lam, **j.keys())

        clean = run()
        spoil(j, 1, 123, head, 9)
        got = run()
        where = touched.any(-1, keepdim=True).expand_as(touched) if norm else touched
        assert torch.equal(~torch.isfinite(got), where)
        assert torch.equal(got[~where], clean[~where])
    # in a prefix: of all its members
    prefixes, tails = [336, 32], [9, 0, 700, 64]
    touched.zero_()
    touched[[0, 2], heads, D + 9] = True
    for norm in (False, True):
        j = Job(4, prefixes + tails, hq, hkv, e4m3, 15, norm=norm)
        front, own = j.tables[:2, :21].contiguous(), j.tables[2:].contiguous()

        def run():
            return pkv.cascade_diff_decode_attention(j.q, j.k, j.v, front, ints(prefixes), ints([0, 2, 3]), ints([2, 0, 3]),
                                                     ints([0, -1, 0, 1]), own, ints(tails), 0.125, j.lam, max_members=2,
                                                     **j.keys())

        clean = run()
        spoil(j, 0, 123, head, 9)
        got = run()
        where = touched.any(-1, keepdim=True).expand_as(touched) if norm else touched
        assert torch.equal(~torch.isfinite(got), where)
        assert torch.equal(got[~where], clean[~where])
    assert pkv.check_device_status() == 0
