"""Ways of calling differential attention: captured and replayed, on two streams, with bad tables and offsets, with no
keys at all, with waits that run out, far in a large pool, and what the binding refuses."""
import math

import pytest
import torch

from diff_helpers import CHUNK_WEIGHT, STEP_WEIGHT, bounds, compare, finish_64, halves, maps_64
from prompt_helpers import make_pool, offsets
from test_gpu_diff import D, Job, check_chunk, check_shared, check_step, ints
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


def calls(pkv, e4m3, seed=0):
    """The three forms, split and not, as functions of an output tensor: [(name, output, call)]."""
    made = []

    def add(name, shape, call, dtype=torch.bfloat16):
        made.append((name, torch.zeros(shape, dtype=dtype, device="cuda"), call))

    lens, ctx = [70, 3, 200], [300, 900, 200]
    a = Job(sum(lens), ctx, 16, 4, e4m3, seed, per_token=True)
    ip, c = ints(offsets(lens)), ints(ctx)
    add("chunk", (sum(lens), 8, 2 * D), lambda out: pkv.paged_diff_prefill_attention(
        a.q, ip, a.k, a.v, a.tables, c, 0.125, a.lam, out, max_context_len=max(ctx), **a.keys()))
    few, far = [2, 1], [9000, 5000]
    f = Job(sum(few), far, 16, 4, e4m3, seed + 1, junk=None)
    fp, fc = ints(offsets(few)), ints(far)
    add("chunk, split", (sum(few), 8, 2 * D), lambda out: pkv.paged_diff_prefill_attention(
        f.q, fp, f.k, f.v, f.tables, fc, 0.125, f.lam, out, max_context_len=max(far), **f.keys()))
    sc = ints([0, 40, 3000])
    s = Job(3, [0, 40, 3000], 16, 4, e4m3, seed + 2)
    add("step", (3, 8, 2 * D), lambda out: pkv.paged_diff_decode_attention(
        s.q, s.k, s.v, s.tables, sc, 0.125, s.lam, out, max_context_len=3000, **s.keys()), torch.float32)
    prefixes, tails = [320, 64], [5, 0, 300, 17, 1]
    j = Job(5, prefixes + tails, 16, 4, e4m3, seed + 3)
    front, own = j.tables[:2].contiguous(), j.tables[2:].contiguous()
    px = (ints(prefixes), ints([0, 3, 4]), ints([4, 0, 2, 1]), ints([0, 1, 0, -1, 0]))
    tc = ints(tails)
    add("shared", (5, 8, 2 * D), lambda out: pkv.cascade_diff_decode_attention(
        j.q, j.k, j.v, front, px[0], px[1], px[2], px[3], own, tc, 0.125, j.lam, out, max_members=3, **j.keys()))
    return made


@pytest.mark.parametrize("e4m3", [False, True])
def test_repeated_calls_give_the_same_bits(pkv, e4m3):
    for name, out, call in calls(pkv, e4m3):
        call(out)
        want = out.clone()
        assert bool(torch.isfinite(want).all()) and want.abs().max() > 0, name
        for _ in range(10):
            out.fill_(7.0)
            call(out)
            assert torch.equal(out, want), name
    assert pkv.check_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_and_replayed(pkv, e4m3):
    """Two graphs of each form, replayed in turns on two streams at a time, give the eager call's bits."""
    for name, out, call in calls(pkv, e4m3):
        call(out)
        want = out.clone()
        torch.cuda.synchronize()
        outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
        for _ in range(2):
            o = torch.empty_like(out)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(o)
            outs.append(o)
            graphs.append(g)
        for _ in range(3):
            for o in outs:
                o.fill_(7.0)
            torch.cuda.synchronize()
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
                    g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, want) for o in outs), name
    assert pkv.check_device_status() == 0


def test_two_streams(pkv):
    """Calls on two streams at once, the stream given or current, share nothing."""
    a, b = calls(pkv, False, 0), calls(pkv, True, 20)
    for (name, x, f), (_, y, g) in zip(a, b):
        f(x), g(y)
        wx, wy = x.clone(), y.clone()
        torch.cuda.synchronize()
        s, t = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(5):
            x.fill_(7.0), y.fill_(7.0)
            torch.cuda.synchronize()
            for _ in range(3):
                with torch.cuda.stream(s):
                    f(x)
                with torch.cuda.stream(t):
                    g(y)
            torch.cuda.synchronize()
            assert torch.equal(x, wx) and torch.equal(y, wy), name
    ctx = [500, 3000]
    j = Job(2, ctx, 8, 2, False, 1)
    want = pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, ints(ctx), 0.125, j.lam, **j.keys())
    torch.cuda.synchronize()
    got = pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, ints(ctx), 0.125, j.lam, stream=s, **j.keys())
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_a_workspace_of_the_callers(pkv):
    ctx = [3000, 70]
    j = Job(2, ctx, 8, 2, False, 1)
    c = ints(ctx)
    need = pkv.diff_decode_workspace_size(2, 8, 2, D, 3000)
    assert need > 0 and pkv.diff_decode_workspace_size(2, 8, 2, D, 64) == 0
    want = pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, c, 0.125, j.lam, max_context_len=3000, **j.keys())
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # any contents
    got = pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, c, 0.125, j.lam, max_context_len=3000, workspace=ws,
                                          **j.keys())
    assert torch.equal(got, want)
    with pytest.raises(pkv.PkvError, match="workspace"):
        pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, c, 0.125, j.lam, max_context_len=3000,
                                        workspace=ws[:need - 256], **j.keys())
    assert pkv.check_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_no_keys_at_all(pkv, e4m3):
    j = Job(3, [16, 0, 0, 0], 8, 2, e4m3, 1)
    own, none = j.tables[1:].contiguous(), ints([0, 0, 0])
    out = torch.full((3, 4, 2 * D), 7.0, device="cuda")
    pkv.paged_diff_decode_attention(j.q, j.k, j.v, own, none, 0.125, j.lam, out, max_context_len=0, **j.keys())
    assert not out.any()
    got = pkv.paged_diff_prefill_attention(j.q, ints([0, 2, 2, 3]), j.k, j.v, own, none, 0.125, j.lam, max_context_len=0,
                                           **j.keys())
    assert not got.any()
    # a prefix and nothing else; a prefix without tokens
    m = maps_64(j.q, [1] * 3, (j.k, j.v), j.scales, [[(j.tables[0], 16)]] * 3, 0.125, j.lam, False)
    pkv.cascade_diff_decode_attention(j.q, j.k, j.v, j.tables[:1].contiguous(), ints([16]), ints([0, 3]), ints([2, 0, 1]),
                                      ints([0, 0, 0]), own, none, 0.125, j.lam, out, max_members=3, max_context_len=0,
                                      **j.keys())
    compare(out, finish_64(m, j.w, j.eps, j.out_scale),
            bounds(m, j.w, j.eps, j.out_scale, STEP_WEIGHT, e4m3, halves(out.dtype)))
    pkv.cascade_diff_decode_attention(j.q, j.k, j.v, j.tables[:1].contiguous(), ints([0]), ints([0, 3]), ints([2, 0, 1]),
                                      ints([0, 0, 0]), own, none, 0.125, j.lam, out, max_members=3, max_context_len=0,
                                      **j.keys())
    assert not out.any()
    # nothing to do
    assert pkv.paged_diff_prefill_attention(j.q[:0], ints([0, 0, 0, 0]), j.k, j.v, own, none, 0.125, j.lam,
                                            **j.keys()).shape == (0, 4, 2 * D)
    assert pkv.paged_diff_decode_attention(j.q[:0], j.k, j.v, own[:0], none[:0], 0.125, j.lam,
                                           **j.keys()).shape == (0, 4, 2 * D)
    assert pkv.check_device_status() == 0


# ------------------------------------------------------------------ bad tables, lengths and offsets

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("far", [False, True])
def test_chunk_bad_ranges(pkv, e4m3, far):
    """Ranges that are wrong are flagged and skipped, the others attended, rows of none left alone."""
    lens = [4, 3, 5]
    ctx = [9000, 5000, 7000] if far else [40, 300, 20]
    j = Job(12, ctx, 8, 2, e4m3, 2, junk=None)
    c = ints(ctx)

    def call(ip):
        out = torch.full((12, 4, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
        pkv.paged_diff_prefill_attention(j.q, ints(ip), j.k, j.v, j.tables, c, 0.125, j.lam, out, **j.keys())
        return out, pkv.check_device_status()

    good, flags = call(offsets(lens))
    assert flags == 0
    for ip, keep in (([0, 4, 7, 13], slice(0, 7)), ([-1, 4, 7, 12], slice(4, 12)), ([0, 4, 2, 2], slice(0, 4))):
        out, flags = call(ip)
        assert flags & pkv.DEVFLAG_BAD_INDPTR, ip
        assert torch.equal(out[keep], good[keep]), ip
        rest = torch.ones(12, dtype=torch.bool, device="cuda")
        rest[keep] = False
        assert bool((out[rest] == 7.0).all()), ip


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_lengths_and_blocks(pkv, e4m3):
    ctx = [40, 100, 64]
    j = Job(3, ctx, 8, 2, e4m3, 5)
    want = pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, ints(ctx), 0.125, j.lam, **j.keys())
    out = pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, ints([40, -3, 64]), 0.125, j.lam, **j.keys())
    assert pkv.check_device_status() == pkv.DEVFLAG_BAD_CONTEXT_LEN
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2]) and not out[1].any()
    out = pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, ints([40, 1 << 30, 64]), 0.125, j.lam, max_context_len=100,
                                          **j.keys())
    assert pkv.check_device_status() == pkv.DEVFLAG_BAD_CONTEXT_LEN and torch.equal(out, want)
    # a block outside the pool reads as zeros: as a sequence whose pool holds zeros there
    bad, zero = j.tables.clone(), j.tables[1, 2].item()
    for wrong in (-5, j.k.shape[0], 1 << 30):
        bad[1, 2] = wrong
        got = [pkv.paged_diff_decode_attention(j.q, j.k, j.v, bad, ints(ctx), 0.125, j.lam, **j.keys()),
               pkv.paged_diff_prefill_attention(j.q, ints([0, 1, 2, 3]), j.k, j.v, bad, ints(ctx), 0.125, j.lam, **j.keys())]
        assert pkv.check_device_status() == pkv.DEVFLAG_BAD_BLOCK_ID
        k, v = j.k.clone(), j.v.clone()
        k.view(torch.uint8)[zero] = 0
        v.view(torch.uint8)[zero] = 0
        assert torch.equal(got[0], pkv.paged_diff_decode_attention(j.q, k, v, j.tables, ints(ctx), 0.125, j.lam, **j.keys()))
        assert torch.equal(got[1], pkv.paged_diff_prefill_attention(j.q, ints([0, 1, 2, 3]), k, v, j.tables, ints(ctx), 0.125,
                                                                    j.lam, **j.keys()))
    assert pkv.check_device_status() == 0


def test_bad_members(pkv):
    """A member outside the batch, offsets that are wrong, lengths past the bound: flagged; sequences that no bad range
    or member belongs to come out right."""
    prefixes, tails = [64, 32], [5, 9, 300, 17]
    j = Job(4, prefixes + tails, 8, 2, False, 3)
    front, own, c = j.tables[:2].contiguous(), j.tables[2:].contiguous(), ints(tails)

    def call(lens=prefixes, ip=(0, 2, 3), who=(0, 2, 1), of=(0, 1, 0, -1), most=2):
        out = pkv.cascade_diff_decode_attention(j.q, j.k, j.v, front, ints(lens), ints(list(ip)), ints(list(who)),
                                                ints(list(of)), own, c, 0.125, j.lam, max_members=most, **j.keys())
        return out, pkv.check_device_status()

    want, flags = call()
    assert flags == 0
    for kw, bits, right in ((dict(who=(0, 9, 1)), pkv.DEVFLAG_BAD_INDPTR, [0, 1, 3]),
                            (dict(who=(0, -1, 1)), pkv.DEVFLAG_BAD_INDPTR, [0, 1, 3]),
                            (dict(ip=(-1, 2, 3)), pkv.DEVFLAG_BAD_INDPTR, [1, 3]),
                            (dict(most=1), pkv.DEVFLAG_BAD_INDPTR, [1, 3]),
                            (dict(lens=[-4, 32]), pkv.DEVFLAG_BAD_CONTEXT_LEN, [1, 3]),
                            # (cut to the table's width, whose entries past the prefix are not its own)
                            (dict(lens=[1 << 20, 32]), pkv.DEVFLAG_BAD_CONTEXT_LEN, [1, 3])):
        got, flags = call(**kw)
        assert flags == bits, kw
        assert torch.equal(got[right], want[right]), kw


# ------------------------------------------------------------------ waits that run out

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,ctx", [([1] * 400, [150 + i % 300 for i in range(400)]),
                                      ([70] * 330, [70 + i % 200 for i in range(330)])], ids=["few", "many"])
def test_waits_run_out_and_the_next_call_is_right(pkv, lens, ctx, e4m3):
    j = Job(sum(lens), ctx, 16, 4, e4m3, 3)
    ip, c = ints(offsets(lens)), ints(ctx)
    out = torch.empty((sum(lens), 8, 2 * D), dtype=torch.bfloat16, device="cuda")

    def call():
        pkv.paged_diff_prefill_attention(j.q, ip, j.k, j.v, j.tables, c, 0.125, j.lam, out, max_context_len=max(ctx), **j.keys())

    pkv.check_device_status()
    call()
    assert pkv.check_device_status() == 0
    want = out.clone()
    with env(PKV_TEST_PREFILL_WAIT_TRIES=2, PKV_TEST_PREFILL_POST_DELAY_CYCLES=40000000):
        call()
        assert pkv.check_device_status() == pkv.DEVFLAG_WAIT_TIMEOUT
    for tries in (1, 3):
        for delay in (100, 1000, 3000, 10000, 20000, 40000, 100000, 1000000):
            out.fill_(7.0)
            with env(PKV_TEST_PREFILL_WAIT_TRIES=tries, PKV_TEST_PREFILL_POST_DELAY_CYCLES=delay):
                call()
            flags = pkv.check_device_status()
            assert flags in (0, pkv.DEVFLAG_WAIT_TIMEOUT)
            if flags == 0:
                assert torch.equal(out, want)
    out.fill_(7.0)
    call()
    assert pkv.check_device_status() == 0
    assert torch.equal(out, want)


# ------------------------------------------------------------------ sizes

@pytest.mark.parametrize("e4m3", [False, True])
def test_many_sequences_and_heads(pkv, e4m3):
    g = torch.Generator().manual_seed(4)
    ctx = torch.randint(0, 200, (300,), generator=g).tolist()
    check_step(pkv, ctx, 8, 4, e4m3)
    lens = [min(c, n) for c, n in zip(ctx, torch.randint(0, 40, (300,), generator=g).tolist())]
    check_chunk(pkv, lens, ctx, 8, 4, e4m3)
    check_step(pkv, [33, 100], 128, 64, e4m3)
    check_chunk(pkv, [33, 100], [50, 333], 128, 64, e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_prefixes(pkv, e4m3):
    """More prefixes than a warp has lanes, most with few members, some with none."""
    g = torch.Generator().manual_seed(6)
    prefixes = [16 * n for n in torch.randint(0, 30, (70,), generator=g).tolist()]
    order, members, at = torch.randperm(120, generator=g).tolist(), [], 0
    for n in torch.randint(0, 3, (70,), generator=g).tolist():
        members.append(order[at:at + n])
        at += n
    tails = torch.randint(0, 60, (120,), generator=g).tolist()
    check_shared(pkv, prefixes, members, tails, 8, 2, e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
def test_blocks_far_into_a_large_pool(pkv, e4m3):
    """Elements past 2^32 of the pool."""
    hkv, blocks, n = 32, 140000, 333
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k, v = (torch.empty((blocks, 16, hkv, D), dtype=dtype, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 32
    ids = ints([blocks - 1 - 3 * i for i in range(21)])
    g = torch.Generator().manual_seed(8)
    for x in (k, v):
        x[ids.long()] = torch.randn((21, 16, hkv, D), generator=g).to(dtype).cuda()
    scales = torch.ones((2, hkv), device="cuda") if e4m3 else None
    q = torch.randn((1, hkv, D), generator=g).to(torch.bfloat16).cuda()
    lam = torch.full((hkv // 2,), 0.4, device="cuda")
    m = maps_64(q, [1], (k, v), scales, [[(ids, n)]], 0.125, lam, False)
    for weight, out in ((STEP_WEIGHT, pkv.paged_diff_decode_attention(q, k, v, ids[None].contiguous(), ints([n]), 0.125, lam,
                                                                      scales=scales)),
                        (CHUNK_WEIGHT[e4m3], pkv.paged_diff_prefill_attention(q, ints([0, 1]), k, v, ids[None].contiguous(),
                                                                              ints([n]), 0.125, lam, scales=scales))):
        compare(out, finish_64(m, None, 0.0, 1.0), bounds(m, None, 0.0, 1.0, weight, e4m3, halves(out.dtype)))
    assert pkv.check_device_status() == 0


def test_scales_of_any_sign(pkv):
    """E4M3 pools whose scales are negative or, of a key head, zero."""
    ctx = [200, 33, 1000]
    for flip in ((0, 0), (0, 1), (1, 1), None):
        j = Job(3, ctx, 8, 4, True, 4)
        if flip is None:
            j.scales[0, 2] = 0.0
        else:
            j.scales[flip] *= -1
        check_step(pkv, ctx, 8, 4, True, job=j)
        check_chunk(pkv, [1, 1, 1], ctx, 8, 4, True, job=j)
        check_shared(pkv, [96], [[1, 0]], [5, 0, 40], 8, 4, True, job=shared_job(flip))


def shared_job(flip):
    j = Job(3, [96, 5, 0, 40], 8, 4, True, 5)
    if flip is None:
        j.scales[0, 2] = 0.0
    else:
        j.scales[flip] *= -1
    return j


@pytest.mark.parametrize("e4m3", [False, True])
def test_one_pair(pkv, e4m3):
    check_step(pkv, [300, 0, 7], 2, 2, e4m3)
    check_chunk(pkv, [140, 3], [200, 7], 2, 2, e4m3, per_token=True)
    check_shared(pkv, [64], [[1, 0]], [5, 0, 40], 2, 2, e4m3)


def test_codes_as_bytes_and_lambda_layouts(pkv):
    ctx = [100, 33]
    j = Job(2, ctx, 8, 2, True, 2)
    c = ints(ctx)
    want = pkv.paged_diff_decode_attention(j.q, j.k, j.v, j.tables, c, 0.125, j.lam, **j.keys())
    for lam in (j.lam, j.lam.expand(2, 4), j.lam.repeat(2, 1), torch.stack((j.lam, j.lam * 0, j.lam), 0)[::2]):
        assert torch.equal(pkv.paged_diff_decode_attention(j.q, j.k.view(torch.uint8), j.v.view(torch.uint8), j.tables, c, 0.125,
                                                           lam, **j.keys()), want)


def test_the_binding_refuses(pkv):
    ctx = [100, 33]
    j = Job(2, ctx, 8, 2, False, 2)
    c, ip = ints(ctx), ints([0, 1, 2])

    def step(**kw):
        a = dict(q=j.q, k=j.k, v=j.v, t=j.tables, c=c, lam=j.lam, out=None, w=j.w, scales=None)
        a.update(kw)
        return pkv.paged_diff_decode_attention(a["q"], a["k"], a["v"], a["t"], a["c"], 0.125, a["lam"], a["out"],
                                               norm_weight=a["w"], scales=a["scales"])

    step()
    for kw, error in ((dict(q=j.q.float()), TypeError), (dict(q=j.q[:, :, :32]), ValueError), (dict(q=j.q[:1]), ValueError),
                      (dict(q=torch.stack((j.q, j.q), 1)[:, 0]), ValueError), (dict(c=c.long()), ValueError),
                      (dict(t=j.tables.long()), TypeError), (dict(lam=j.lam.double()), TypeError),
                      (dict(lam=j.lam[:3]), ValueError), (dict(lam=j.lam.expand(3, 4)), ValueError),
                      (dict(lam=j.lam.repeat(2, 2)[:, ::2]), ValueError), (dict(lam=j.lam.cpu()), ValueError),
                      (dict(lam=None), TypeError), (dict(w=j.w[:64]), ValueError), (dict(w=j.w.float()), ValueError),
                      (dict(out=torch.empty((2, 4, 2 * D), dtype=torch.half, device="cuda")), ValueError),
                      (dict(out=torch.empty((2, 8, D), dtype=torch.bfloat16, device="cuda")), ValueError),
                      (dict(scales=torch.ones((2, 2), device="cuda")), pkv.PkvError), (dict(out=j.q.view(2, 4, 2 * D)), pkv.PkvError)):
        with pytest.raises(error):
            step(**kw)
    with pytest.raises(ValueError):  # fp32 is for one token's forms
        pkv.paged_diff_prefill_attention(j.q, ip, j.k, j.v, j.tables, c, 0.125, j.lam,
                                         torch.empty((2, 4, 2 * D), device="cuda"))
    with pytest.raises(pkv.PkvError, match="head_dim"):
        k, v, _, t = make_pool([40], 2, 128, False, 1)
        pkv.paged_diff_decode_attention(torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda"), k, v, t, ints([40]), 0.1,
                                        j.lam[:2])
    assert pkv.check_device_status() == 0
