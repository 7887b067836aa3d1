"""Ways of calling the prompt side that its documents allow: captured and replayed chains, side streams, empty calls,
tables far wider than the contexts, many sequences, many heads, E4M3 pools as bytes."""
import math

import pytest
import torch

from prompt_helpers import BF16_HALF, attention_64, attention_bounds, make_pool, offsets, rope_64

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


def normal(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


class Chain:
    """A chunk written, attended and read back, over buffers that stay."""

    def __init__(self, pkv, lens, past, e4m3, seed, hq=16, hkv=4, d=128):
        self.pkv, self.lens, self.ctx = pkv, lens, [n + p for n, p in zip(lens, past)]
        self.hq, self.hkv, self.d = hq, hkv, d
        self.k, self.v, self.scales, self.tables = make_pool(self.ctx, hkv, d, e4m3, seed)
        g = torch.Generator().manual_seed(seed)
        T = sum(lens)
        self.packed = normal(g, T, hq + 2 * hkv, d)
        self.pos = ints([p + i for n, p in zip(lens, past) for i in range(n)])
        b = torch.tensor([b for b, n in enumerate(lens) for _ in range(n)], device="cuda", dtype=torch.long)
        self.slots = (self.tables[b, self.pos.long() // 16].long() * 16 + self.pos % 16).contiguous()
        self.ip, self.c, self.kv_ip = ints(offsets(lens)), ints(self.ctx), ints(offsets(self.ctx))
        self.f, _ = pkv.rope_inv_freq(d, device="cuda")
        self.q, self.out = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda"), None
        self.ko, self.vo = (torch.empty((sum(self.ctx), hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def run(self, stream=None):
        p, (q, k, v) = self.pkv, self.packed.split((self.hq, self.hkv, self.hkv), 1)
        p.qk_norm_rope_append(q, k, v, self.pos, self.slots, self.k, self.v, self.q, inv_freq=self.f, scales=self.scales,
                              stream=stream)
        self.out = p.paged_prefill_attention(self.q, self.ip, self.k, self.v, self.tables, self.c, 0.1, self.out,
                                             scales=self.scales, stream=stream)
        p.paged_kv_gather(self.k, self.v, self.tables, self.kv_ip, self.ko, self.vo, scales=self.scales, stream=stream)

    def result(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (self.q, self.out, self.ko, self.vo, self.k.view(torch.uint8), self.v.view(torch.uint8))]

    def check(self):
        """The last run's attention against the definition over the pool as it is."""
        ref, _, mag, size = attention_64(self.q, self.lens, self.k, self.v, self.scales, self.tables, self.ctx, 0.1, True)
        bound, _ = attention_bounds(ref, mag, size, self.q, self.scales is not None, self.d)
        assert float(((self.out.double() - ref).abs() - bound).max()) <= 0


CHUNKS = [([1, 3, 7], [900, 40, 0]), ([300, 5, 90], [0, 700, 33])]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,past", CHUNKS)
def test_chain_captured_and_replayed_on_other_data(pkv, lens, past, e4m3):
    a = Chain(pkv, lens, past, e4m3, 1)
    a.run()  # makes the output
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for seed in (2, 3):
        g = torch.Generator().manual_seed(seed)
        a.packed.copy_(normal(g, *a.packed.shape))
        a.pos.copy_(a.pos + seed)
        start = a.k.clone(), a.v.clone()
        for x in (a.q, a.out, a.ko, a.vo):
            x.fill_(7.0)
        graph.replay()
        got = a.result()
        a.check()
        a.k.copy_(start[0]), a.v.copy_(start[1])
        a.run()
        for x, y in zip(got, a.result()):
            assert torch.equal(x, y)
    assert pkv.check_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_chains_on_two_streams(pkv, e4m3):
    chains = [Chain(pkv, *CHUNKS[i], e4m3, 5 + i) for i in range(2)]
    wants = []
    for c in chains:
        c.run()
        wants.append(c.result())
        c.check()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(8):
        for c, s in zip(chains, streams):
            c.run(stream=s)
    for c, want in zip(chains, wants):
        for x, y in zip(c.result(), want):
            assert torch.equal(x, y)
    assert pkv.check_device_status() == 0


def test_empty_calls(pkv):
    k, v, _, tables = make_pool([40], 2, 64, False, 1)
    was = k.clone()
    e = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0,), dtype=torch.int64, device="cuda")
    assert pkv.qk_norm_rope_append(e, e[:, :2], e[:, :2], None, none, k, v).shape == (0, 8, 64)
    assert pkv.paged_prefill_attention(e, ints([0, 0]), k, v, tables, ints([40]), 0.1).shape == (0, 8, 64)
    q = torch.full((5, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    pkv.paged_prefill_attention(q, ints([0]), k, v, tables[:0], ints([]), 0.1, out)  # rows of no sequence
    pkv.paged_prefill_attention(q, ints([0, 0]), k, v, tables, ints([40]), 0.1, out)
    ko, vo = (torch.full((5, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.paged_kv_gather(k, v, tables, ints([2, 2]), ko, vo)
    pkv.paged_kv_gather(k, v, tables[:0], ints([0]), ko, vo)
    pkv.paged_kv_gather(k, v, tables, ints([0, 0]), ko[:0], vo[:0])
    assert pkv.check_device_status() == 0
    assert torch.equal(k, was) and all(bool((x == 7).all()) for x in (out, ko, vo))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("capacity", [8192, 131072, 1 << 20])
@pytest.mark.parametrize("lens,ctx", [([1], [777]), ([5, 0, 1, 8], [1800, 900, 1, 700]), ([257, 33, 600], [257, 1033, 1100])])
def test_tables_of_the_models_limit(pkv, lens, ctx, capacity, e4m3):
    """Tables as wide as the longest context allowed, and no max_context_len: as in a captured step."""
    hq, hkv, d = 16, 4, 128
    k, v, scales, tables = make_pool(ctx, hkv, d, e4m3, 3, junk=math.nan)
    g = torch.Generator().manual_seed(capacity + len(lens))
    q = normal(g, sum(lens), hq, d)
    wide = torch.full((len(lens), capacity // 16), k.shape[0] - 1, dtype=torch.int32, device="cuda")
    wide[:, :tables.shape[1]] = tables
    lse = torch.empty(q.shape[:2], device="cuda")
    out = pkv.paged_prefill_attention(q, ints(offsets(lens)), k, v, wide, ints(ctx), 0.1, lse=lse, scales=scales)
    assert pkv.check_device_status() == 0
    ref, ref_lse, mag, size = attention_64(q, lens, k, v, scales, tables, ctx, 0.1, True)
    bound, lse_bound = attention_bounds(ref, mag, size, q, e4m3, d)
    assert float(((out.double() - ref).abs() - bound).max()) <= 0
    assert float(((lse.double() - ref_lse).abs() - ref_lse.abs() * 2.0 ** -22).max()) <= lse_bound


@pytest.mark.parametrize("e4m3", [False, True])
def test_thousands_of_sequences(pkv, e4m3):
    g = torch.Generator().manual_seed(9)
    n, hq, hkv, d = 4000, 4, 2, 64
    lens = torch.randint(0, 3, (n,), generator=g).tolist()
    ctx = [x + int(c) for x, c in zip(lens, torch.randint(0, 40, (n,), generator=g))]
    k, v, scales, tables = make_pool(ctx, hkv, d, e4m3, 4)
    q = normal(g, sum(lens), hq, d)
    out = pkv.paged_prefill_attention(q, ints(offsets(lens)), k, v, tables, ints(ctx), 0.125, scales=scales)
    assert pkv.check_device_status() == 0
    ref, _, mag, size = attention_64(q, lens, k, v, scales, tables, ctx, 0.125, True)
    bound, _ = attention_bounds(ref, mag, size, q, e4m3, d)
    assert float(((out.double() - ref).abs() - bound).max()) <= 0
    rows = sum(ctx)
    ko, vo = (torch.empty((rows, hkv, d), device="cuda") for _ in range(2))
    pkv.paged_kv_gather(k, v, tables, ints(offsets(ctx)), ko, vo, scales=scales)
    b = torch.repeat_interleave(torch.arange(n), torch.tensor(ctx)).cuda()
    at = torch.cat([torch.arange(c) for c in ctx]).cuda()
    for i, (x, o) in enumerate(((k, ko), (v, vo))):
        want = x[tables[b, at // 16].long(), at % 16].float()
        assert torch.equal(o, want if scales is None else want * scales[i][:, None])


@pytest.mark.parametrize("T,hq,hkv,d,rot", [(3, 4096, 4096, 64, 64), (5, 257, 1, 128, 128), (40, 1, 131, 64, 16)])
def test_many_heads(pkv, T, hq, hkv, d, rot):
    g = torch.Generator().manual_seed(hq)
    q, k, v = normal(g, T, hq, d), normal(g, T, hkv, d), normal(g, T, hkv, d)
    w = (1 + 0.2 * torch.randn((2, d), generator=g)).to(torch.bfloat16).cuda()
    pos, slots = torch.arange(T, dtype=torch.int32, device="cuda") * 11, torch.arange(T, device="cuda") + 3
    kc, vc = (torch.zeros((4, 16, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    f, _ = pkv.rope_inv_freq(rot, device="cuda")
    out = pkv.qk_norm_rope_append(q, k, v, pos, slots, kc, vc, q_weight=w[0], k_weight=w[1], inv_freq=f)
    for got, x, wt in ((out, q, w[0]), (kc.view(-1, hkv, d)[slots], k, w[1])):
        want = rope_64(x, wt, 1e-6, pos, f, False, 1.0)
        # fp32 steps below 40 roundings of 2^-24 of the row's largest, the angle 2^-22, one rounding to bf16
        size = want.abs().amax(-1, keepdim=True) * 2
        assert bool(((got.double() - want).abs() <= BF16_HALF * want.abs() + 2.0 ** -18 * size).all())
    ko, vo = (torch.empty((T, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.paged_kv_gather(kc, vc, ints([[0, 1, 2, 3]]), ints([0, T]), ko, vo, starts=ints([3]))
    assert torch.equal(ko, kc.view(-1, hkv, d)[slots]) and torch.equal(vo, v)
    assert pkv.check_device_status() == 0


def test_e4m3_pools_as_bytes(pkv):
    a, b = Chain(pkv, *CHUNKS[0], True, 8), Chain(pkv, *CHUNKS[0], True, 8)
    b.k, b.v = b.k.view(torch.uint8), b.v.view(torch.uint8)
    a.run(), b.run()
    for x, y in zip(a.result(), b.result()):
        assert torch.equal(x, y)
