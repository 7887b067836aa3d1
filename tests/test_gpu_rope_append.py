"""Norm + rotation + append in one pass against the definition in 64 bits, and reading pages
back: layouts, part of the head, far positions, strides, padding, E4M3 pools, bad slots."""
import math

import pytest
import torch

from prompt_helpers import BF16_HALF, E4M3_HALF, make_pool, offsets, rope_64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


def inputs(T, hq, hkv, d, seed, far=100000):
    g = torch.Generator().manual_seed(seed)
    packed = (torch.randn((T, hq + 2 * hkv, d), generator=g) * 1.3).to(torch.bfloat16).cuda()
    pos = torch.randint(0, far, (T,), generator=g).to(torch.int32).cuda()
    w = (1 + 0.3 * torch.randn((2, d), generator=g)).to(torch.bfloat16).cuda()
    return packed, pos, w


# fp32 steps of norm and rotation: the sum of D squares (D/16 in a thread, then a tree), the root
# (2 ulp), four products and a sum, sine and cosine (2 ulp): below 40 roundings of 2^-24 relative to
# the pair's size; the angle in half turns is off by 2^-25 of a turn at most 2^-22 rad
ARITH = 40 * 2.0 ** -24 + 2.0 ** -22


def near(got, want, size, half):
    """Rounded once: |got - want| <= half |want| (+ what the arithmetic may be off, of the pair's size)."""
    bound = half * (want.abs() + ARITH * size) + ARITH * size
    off = (got.double() - want).abs() - bound
    assert float(off.max()) <= 0, float((got.double() - want).abs().max())


def pair_size(x, w, eps):
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    return x.abs().amax(-1, keepdim=True) * math.sqrt(2)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,rot,interleaved,norm", [
    (1, 8, 2, 64, 64, False, True),
    (1, 32, 8, 128, 128, True, False),
    (7, 8, 8, 64, 16, False, False),
    (64, 32, 8, 128, 128, False, True),
    (333, 16, 2, 128, 64, False, True),
    (333, 8, 1, 64, 32, True, True),
    (1000, 5, 3, 128, 112, False, False),
    (2049, 8, 2, 64, 0, False, True),
    (5000, 64, 8, 128, 96, True, True),
])
def test_matches_definition(pkv, T, hq, hkv, d, rot, interleaved, norm, e4m3):
    packed, pos, w = inputs(T, hq, hkv, d, T + rot)
    q, k, v = packed.split((hq, hkv, hkv), 1)
    kc, vc, scales, _ = make_pool([T], hkv, d, e4m3, T)
    before = kc.clone(), vc.clone()
    g = torch.Generator().manual_seed(T + 5)
    slots = torch.randperm(kc.shape[0] * 16, generator=g)[:T].cuda()
    slots[1::5] = -1  # padding tokens
    inv_freq, rope_scale = pkv.rope_inv_freq(rot, 500000.0, scaling="yarn", factor=8.0, device="cuda") if rot else (None, 1.0)
    wq, wk = (w[0], w[1]) if norm else (None, None)
    pkv.check_device_status()
    out = pkv.qk_norm_rope_append(q, k, v, pos if rot else None, slots, kc, vc, q_weight=wq, k_weight=wk, eps=1e-5,
                                  inv_freq=inv_freq, interleaved=interleaved, rope_scale=rope_scale, scales=scales)
    assert pkv.check_device_status() == 0
    near(out, rope_64(q, wq, 1e-5, pos, inv_freq, interleaved, rope_scale),
         pair_size(q, wq, 1e-5) * rope_scale, BF16_HALF)
    kept = slots >= 0
    want_k = rope_64(k, wk, 1e-5, pos, inv_freq, interleaved, rope_scale)[kept]
    size_k = (pair_size(k, wk, 1e-5) * rope_scale)[kept]
    rows = slots[kept]
    if e4m3:
        sk = scales[0].double()[:, None]
        got = kc.view(-1, hkv, d).view(torch.uint8)[rows].view(torch.float8_e4m3fn).double()
        w64 = want_k / sk
        bound = torch.maximum(E4M3_HALF * w64.abs(), torch.full_like(w64, 2.0 ** -10)) + 2 * ARITH * size_k / sk
        sat = w64.abs() > 448
        off = (got - w64.clamp(-448, 448)).abs() - bound
        assert float(off.max()) <= 0 and bool((got[sat].abs() == 448).all())
        code = (v[kept].float() / scales[1][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(vc.view(-1, hkv, d).view(torch.uint8)[rows], code)
    else:
        near(kc.view(-1, hkv, d)[rows], want_k, size_k, BF16_HALF)
        assert torch.equal(vc.view(-1, hkv, d)[rows], v[kept])
    rest = torch.ones(kc.shape[0] * 16, dtype=torch.bool, device="cuda")
    rest[rows] = False
    for now, was in zip((kc, vc), before):
        assert torch.equal(now.view(torch.uint8).view(rest.numel(), -1)[rest], was.view(torch.uint8).view(rest.numel(), -1)[rest])


def test_equals_append_without_norm_and_rotation(pkv):
    for e4m3 in (False, True):
        packed, _, _ = inputs(100, 8, 2, 128, 3)
        q, k, v = packed.split((8, 2, 2), 1)
        k, v = k.contiguous(), v.contiguous()
        k[3, 1, 5] = math.nan
        v[4, 0, 6] = math.inf
        kc, vc, scales, _ = make_pool([100], 2, 128, e4m3, 4)
        kd, vd = kc.clone(), vc.clone()
        slots = torch.randperm(112, device="cuda")[:100]
        out = pkv.qk_norm_rope_append(q, k, v, None, slots, kc, vc, scales=scales)
        pkv.paged_kv_append(k, v, slots, kd, vd, scales=scales)
        assert torch.equal(out, q)
        for a, b in ((kc, kd), (vc, vd)):
            if e4m3:
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            else:
                assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(0), b.nan_to_num(0))


@pytest.mark.parametrize("scale", [1.0, 0.015625, 0.0117, 3.0, 1e-3, 7e37, 1e-39])
def test_codes_are_those_of_the_append(pkv, scale):
    """Values at and next to every border of two codes, under scales that divide exactly or not."""
    hkv, d = 2, 128
    codes = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (codes[1:] + codes[:-1]) / 2
    x = torch.cat([codes, mid, mid * (1 + 2 ** -7), mid * (1 - 2 ** -7), torch.tensor([449.0, 464.0, 470.0, 1e4])])
    x = torch.cat([x, -x]).double() * scale
    x = x.clamp(-3e38, 3e38).to(torch.bfloat16)
    T = (x.numel() + hkv * d - 1) // (hkv * d)
    k = torch.zeros(T * hkv * d, dtype=torch.bfloat16)
    k[: x.numel()] = x
    k = k.view(T, hkv, d).cuda()
    v = k.flip(0).contiguous()
    q = torch.zeros((T, 2, d), dtype=torch.bfloat16, device="cuda")
    kc, vc, scales, _ = make_pool([T], hkv, d, True, 4)
    scales.fill_(scale)
    kd, vd = kc.clone(), vc.clone()
    slots = torch.arange(T, device="cuda")
    pkv.qk_norm_rope_append(q, k, v, None, slots, kc, vc, scales=scales)
    pkv.paged_kv_append(k, v, slots, kd, vd, scales=scales)
    assert torch.equal(kc.view(torch.uint8), kd.view(torch.uint8)) and torch.equal(vc.view(torch.uint8), vd.view(torch.uint8))


def test_in_place_and_strided_output(pkv):
    packed, pos, w = inputs(77, 8, 2, 64, 9)
    kc, vc, _, _ = make_pool([77], 2, 64, False, 1)
    slots = torch.arange(77, device="cuda")
    f, _ = pkv.rope_inv_freq(64, device="cuda")
    q, k, v = packed.split((8, 2, 2), 1)
    want = pkv.qk_norm_rope_append(q, k, v, pos, slots, kc, vc, q_weight=w[0], k_weight=w[1], inv_freq=f)
    k2, v2 = kc.clone(), vc.clone()
    p2 = packed.clone()
    q2, kk, vv = p2.split((8, 2, 2), 1)
    got = pkv.qk_norm_rope_append(q2, kk, vv, pos, slots, k2, v2, q2, q_weight=w[0], k_weight=w[1], inv_freq=f)
    assert got.data_ptr() == q2.data_ptr() and torch.equal(q2, want)
    assert torch.equal(p2[:, 8:], packed[:, 8:]) and torch.equal(k2, kc) and torch.equal(v2, vc)


def test_far_positions(pkv):
    """Angles of positions up to 2^31 - 1."""
    T, d = 64, 128
    packed, _, _ = inputs(T, 4, 1, d, 2)
    q, k, v = packed.split((4, 1, 1), 1)
    pos = torch.randint(2 ** 30, 2 ** 31 - 1, (T,), dtype=torch.int64).to(torch.int32).cuda()
    pos[0] = 2 ** 31 - 1
    f, _ = pkv.rope_inv_freq(d, device="cuda")
    kc, vc, _, _ = make_pool([T], 1, d, False, 1)
    out = pkv.qk_norm_rope_append(q, k, v, pos, torch.arange(T, device="cuda"), kc, vc, inv_freq=f)
    # the angle's product of 2^31 and f in fp64 is off by 2^-53 of up to 2^31, here and there
    want = rope_64(q, None, 0, pos, f, False, 1.0)
    off = (out.double() - want).abs() - BF16_HALF * want.abs() - 2.0 ** -18 * pair_size(q, None, 0)
    assert float(off.max()) <= 0


def test_bad_slots(pkv):
    packed, pos, _ = inputs(20, 4, 1, 64, 2)
    q, k, v = packed.split((4, 1, 1), 1)
    kc, vc, _, _ = make_pool([20], 1, 64, False, 1)
    was = kc.clone()
    slots = torch.full((20,), -1, device="cuda", dtype=torch.int64)
    slots[7] = kc.shape[0] * 16
    pkv.check_device_status()
    out = pkv.qk_norm_rope_append(q, k, v, None, slots, kc, vc)
    assert pkv.check_device_status() == pkv.DEVFLAG_BAD_SLOT
    assert torch.equal(kc, was) and torch.equal(out, q)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,hkv,d", [([1], 1, 64), ([5, 0, 16, 33], 2, 64), ([1000], 8, 128), ([3] * 700, 3, 128),
                                        ([513, 1, 2000], 8, 128)])
def test_gather(pkv, lens, hkv, d, e4m3, fp32):
    k, v, scales, tables = make_pool(lens, hkv, d, e4m3, len(lens))
    total = sum(lens)
    dtype = torch.float32 if fp32 else torch.bfloat16
    ko, vo = (torch.full((total + 5, hkv, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    starts = torch.tensor([min(2, n) for n in lens], dtype=torch.int32, device="cuda")
    take = [n - min(2, n) for n in lens]
    for st, ns in ((None, lens), (starts, take)):
        ip = torch.tensor(offsets(ns), dtype=torch.int32, device="cuda")
        ko.fill_(7.0), vo.fill_(7.0)
        pkv.check_device_status()
        pkv.paged_kv_gather(k, v, tables, ip, ko, vo, starts=st, scales=scales)
        assert pkv.check_device_status() == 0
        for i, (x, o) in enumerate(((k, ko), (v, vo))):
            rows = [x[tables[b, : (n + 15) // 16].long()].flatten(0, 1)[:n] for b, n in enumerate(lens)]
            rows = torch.cat([r[len(r) - m:] for r, m in zip(rows, ns)]).float()
            if e4m3:
                rows = rows * scales[i][:, None]  # one fp32 product
            assert torch.equal(o[: sum(ns)], rows.to(dtype))
            assert bool((o[sum(ns):] == 7).all())


def test_gather_bad_data(pkv):
    lens = [40, 50]
    k, v, _, tables = make_pool(lens, 2, 64, False, 3)
    ko, vo = (torch.full((90, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ip = torch.tensor(offsets(lens), dtype=torch.int32, device="cuda")
    t = tables.clone()
    t[0, 1] = -3
    pkv.paged_kv_gather(k, v, t, ip, ko, vo)
    assert pkv.check_device_status() == pkv.DEVFLAG_BAD_BLOCK_ID
    assert bool((ko[16:32] == 0).all()) and not bool((ko[:16] == 0).any(-1).all())
    starts = torch.tensor([30, -1], dtype=torch.int32, device="cuda")
    pkv.paged_kv_gather(k, v, tables, ip, ko, vo, starts=starts)
    assert pkv.check_device_status() & pkv.DEVFLAG_BAD_CONTEXT_LEN
    assert bool((vo[40] == 0).all()) and bool((ko[34:40] == 0).all())
    ko.fill_(7)
    ip[2] = 1000
    pkv.paged_kv_gather(k, v, tables, ip, ko, vo)
    assert pkv.check_device_status() & pkv.DEVFLAG_BAD_INDPTR


def test_gather_bad_ranges_leave_their_rows(pkv):
    """A range that ends before it starts has no row to find it by, and one past the last row has: both are
    flagged, and only the rows of good ranges are written."""
    lens = [40, 50, 30]
    k, v, _, tables = make_pool(lens, 2, 64, False, 4)
    ref_k, ref_v = (torch.empty((120, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.paged_kv_gather(k, v, tables, torch.tensor(offsets(lens), dtype=torch.int32, device="cuda"), ref_k, ref_v)
    assert pkv.check_device_status() == 0
    for ip, good in (([0, 40, 30, 30], 40), ([0, 40, 90, 121], 90), ([0, 40, 90, 85], 90)):
        ko, vo = (torch.full((120, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pkv.paged_kv_gather(k, v, tables, torch.tensor(ip, dtype=torch.int32, device="cuda"), ko, vo)
        assert pkv.check_device_status() == pkv.DEVFLAG_BAD_INDPTR
        for got, ref in ((ko, ref_k), (vo, ref_v)):
            if ip[2] == 90:
                assert torch.equal(got[:good], ref[:good])
            assert bool((got[max(ip):] == 7).all()) and (ip[3] != 121 or bool((got[90:] == 7).all()))


def test_prompt_to_decode(pkv):
    """A prompt in two chunks (norm + rotation + append, then attention), a decode step on the
    same pool, and the pages read back: the whole path against one pass in 64 bits."""
    from prompt_helpers import attention_64, attention_bounds

    hq, hkv, d, total = 8, 2, 128, 300
    kc, vc, _, tables = make_pool([total + 1], hkv, d, False, 8)
    packed, _, w = inputs(total + 1, hq, hkv, d, 12)
    f, _ = pkv.rope_inv_freq(d, device="cuda")
    slot = (tables[0].long()[:, None] * 16 + torch.arange(16, device="cuda")).view(-1)[: total + 1].contiguous()
    outs, qs = [], []
    scale = 1 / math.sqrt(d)
    for a, b in ((0, 177), (177, total), (total, total + 1)):
        q, k, v = packed[a:b].split((hq, hkv, hkv), 1)
        pos = torch.arange(a, b, dtype=torch.int32, device="cuda")
        q = pkv.qk_norm_rope_append(q, k, v, pos, slot[a:b].contiguous(), kc, vc, q_weight=w[0], k_weight=w[1], inv_freq=f)
        ctx = torch.tensor([b], dtype=torch.int32, device="cuda")
        if b - a > 1:
            o = pkv.paged_prefill_attention(q, torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), kc, vc, tables,
                                            ctx, scale)
        else:
            o = pkv.paged_decode_attention(q, kc, vc, tables, ctx, scale)
        outs.append(o), qs.append(q)
    ko, vo = (torch.empty((total + 1, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.paged_kv_gather(kc, vc, tables, torch.tensor([0, total + 1], dtype=torch.int32, device="cuda"), ko, vo)
    assert pkv.check_device_status() == 0
    q, out = torch.cat(qs), torch.cat(outs)
    assert torch.equal(vo, packed[:, hq + hkv:])
    near(ko, rope_64(packed[:, hq:hq + hkv], w[1], 1e-6, torch.arange(total + 1, device="cuda"), f, False, 1.0),
         pair_size(packed[:, hq:hq + hkv], w[1], 1e-6), BF16_HALF)
    ref, _, mag, size = attention_64(q, [total + 1], kc, vc, None, tables, [total + 1], scale, True)
    bound, _ = attention_bounds(ref, mag, size, q, False, d)
    assert float(((out.double() - ref).abs() - bound).max()) <= 0
