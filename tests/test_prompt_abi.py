"""The prompt side's calls without a GPU: refusals by the C ABI before any CUDA call, refusals by
the binding, and the rotation's frequencies against their definitions."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


def desc(pkv, **kw):
    base = dict(k_cache=0x10000, v_cache=0x20000, num_blocks=64, block_size=16, num_kv_heads=2, head_dim=64,
                kv_dtype=0, scales=None)
    base.update(kw)
    return pkv.CacheDesc(**base)


def last(pkv):
    return pkv.lib.pkv_last_error().decode()


def prefill(pkv, d, q=0x60000, stride=512, indptr=0x50000, T=10, tables=0x80000, blocks=7, lens=0x90000, B=4, hq=8,
            max_len=100, causal=1, scale=0.125, out=0x70000, lse=None):
    return pkv.lib.pkv_paged_prefill_attention(ctypes.byref(d), q, stride, indptr, T, tables, blocks, lens, B, hq, max_len,
                                               causal, scale, out, lse, None, 0, None)


def test_prefill_refusals(pkv):
    bad, unsup = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED
    d = desc(pkv)
    assert prefill(pkv, d, B=0) == pkv.PKV_OK and prefill(pkv, d, T=0) == pkv.PKV_OK  # nothing to do, no CUDA call
    assert prefill(pkv, desc(pkv, head_dim=96)) == unsup
    assert prefill(pkv, desc(pkv, block_size=32)) == unsup
    assert prefill(pkv, desc(pkv, kv_dtype=1)) == bad and "scales" in last(pkv)
    assert prefill(pkv, d, hq=6) == unsup and "group" in last(pkv)
    assert prefill(pkv, d, hq=5) == bad
    assert prefill(pkv, d, hq=32) == unsup  # a query group of 16
    assert prefill(pkv, d, T=-1) == bad and prefill(pkv, d, B=-1) == bad and prefill(pkv, d, B=70000) == bad
    assert prefill(pkv, d, q=None) == bad and prefill(pkv, d, q=0x60008) == bad
    assert prefill(pkv, d, stride=504) == bad and "stride" in last(pkv)  # less than a token's heads
    assert prefill(pkv, d, stride=513) == bad
    for name in ("indptr", "tables", "lens", "out"):
        assert prefill(pkv, d, **{name: None}) == bad
    assert prefill(pkv, d, out=0x70008) == bad and prefill(pkv, d, lse=0x70001) == bad
    assert prefill(pkv, d, max_len=113) == bad and "max_blocks_per_seq" in last(pkv)
    assert prefill(pkv, d, max_len=-1) == bad and prefill(pkv, d, blocks=0, max_len=0) == bad
    assert prefill(pkv, d, max_len=(1 << 30) + 1, blocks=1 << 27) == unsup
    assert prefill(pkv, d, causal=2) == bad
    for scale in (float("nan"), float("inf"), 2e38):
        assert prefill(pkv, d, scale=scale) == bad
    assert pkv.lib.pkv_prefill_workspace_size(4, 10, 6, 2, 64, 100) == 0 and "group" in last(pkv)
    assert pkv.lib.pkv_prefill_workspace_size(0, 10, 8, 2, 64, 100) == 0


def append(pkv, d, **kw):
    a = dict(q=0x30000, k=0x40000, v=0x50000, q_stride=512, k_stride=128, v_stride=128, positions=0x60000,
             slot_mapping=0x70000, num_tokens=4, num_q_heads=8, rotary_dim=64, interleaved=0, rope_scale=1.0,
             inv_freq=0x80000, q_weight=None, k_weight=None, eps=1e-6, q_out=0x900000, q_out_stride=512)
    a.update(kw)
    from paged_kv_cache_17_gb300.prompt import RopeAppendDesc

    x = RopeAppendDesc(**a)
    return pkv.lib.pkv_qk_norm_rope_append(ctypes.byref(d), ctypes.byref(x), None)


def test_append_refusals(pkv):
    bad, unsup = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED
    d = desc(pkv)
    assert append(pkv, d, num_tokens=0) == pkv.PKV_OK
    assert append(pkv, d, num_tokens=-1) == bad and append(pkv, d, num_tokens=1 << 31) == bad
    assert pkv.lib.pkv_qk_norm_rope_append(ctypes.byref(d), None, None) == bad
    assert append(pkv, desc(pkv, head_dim=80)) == unsup
    assert append(pkv, d, num_q_heads=0) == bad and append(pkv, d, num_q_heads=5000) == unsup
    for rot in (8, 24, -16, 80):
        assert append(pkv, d, rotary_dim=rot) == unsup and "rotary_dim" in last(pkv)
    assert append(pkv, d, interleaved=2) == bad
    assert append(pkv, d, rope_scale=float("nan")) == bad
    assert append(pkv, d, q_weight=0x100000, eps=-1.0) == bad and append(pkv, d, k_weight=0x100000, eps=float("nan")) == bad
    assert append(pkv, d, q_weight=0x100008) == bad
    for name in ("q", "k", "v", "q_out", "slot_mapping", "positions", "inv_freq"):
        assert append(pkv, d, **{name: None}) == bad
    for name in ("q", "k", "v", "q_out"):
        assert append(pkv, d, **{name: 0x30008}) == bad and name in last(pkv)
    assert append(pkv, d, k_stride=120) == bad and append(pkv, d, v_stride=129) == bad
    assert append(pkv, d, q_out=0x30000 + 512, q_out_stride=512) == bad and "overlaps" in last(pkv)
    assert append(pkv, d, q_out=0x30000, q_out_stride=1024) == bad  # q itself, at another stride


def gather(pkv, d, tables=0x80000, blocks=7, indptr=0x50000, starts=None, B=4, rows=10, k=0x60000, v=0x70000, dt=0):
    return pkv.lib.pkv_paged_kv_gather(ctypes.byref(d), tables, blocks, indptr, starts, B, rows, k, v, dt, None)


def test_gather_refusals(pkv):
    bad = pkv.PKV_ERR_INVALID_ARG
    d = desc(pkv)
    assert gather(pkv, d, B=0) == pkv.PKV_OK and gather(pkv, d, rows=0) == pkv.PKV_OK
    assert gather(pkv, d, B=-1) == bad and gather(pkv, d, rows=-1) == bad and gather(pkv, d, rows=1 << 31) == bad
    assert gather(pkv, d, blocks=0) == bad and gather(pkv, d, dt=2) == bad
    for name in ("tables", "indptr", "k", "v"):
        assert gather(pkv, d, **{name: None}) == bad
    assert gather(pkv, d, k=0x60008) == bad and gather(pkv, d, v=0x70004) == bad and gather(pkv, d, starts=0x3) == bad
    assert gather(pkv, desc(pkv, head_dim=32)) == pkv.PKV_ERR_UNSUPPORTED


def test_binding_refuses_tensors_that_are_not_on_a_gpu(pkv):
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.paged_prefill_attention(q, i, k, k.clone(), t, i[:1], 0.1)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.paged_kv_gather(k, k.clone(), t, i, q, q)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.qk_norm_rope_append(q, q, q, None, i.long(), k, k.clone())
    with pytest.raises(TypeError):
        pkv.paged_kv_gather(None, k, t, i, q, q)


def test_rope_frequencies(pkv):
    f, scale = pkv.rope_inv_freq(64, 10000.0)
    assert scale == 1.0 and f.dtype == torch.float64
    p = torch.arange(32, dtype=torch.float64)
    plain = 10000.0 ** (-p / 32)
    assert torch.allclose(f, plain, rtol=1e-15)
    f, _ = pkv.rope_inv_freq(64, 10000.0, scaling="linear", factor=4.0)
    assert torch.allclose(f, plain / 4, rtol=1e-15)
    f, _ = pkv.rope_inv_freq(64, 10000.0, scaling="ntk", factor=4.0)
    assert f[0] == 1.0 and math.isclose(float(f[-1]), float(plain[-1]) / 4, rel_tol=1e-12)
    f, _ = pkv.rope_inv_freq(64, 500000.0, scaling="banded", factor=8.0, original_max_position=8192)
    plain = 500000.0 ** (-p / 32)
    wave = 2 * math.pi / plain
    assert torch.equal(f[wave < 8192 / 4], plain[wave < 8192 / 4])
    assert torch.allclose(f[wave > 8192], plain[wave > 8192] / 8, rtol=1e-15)
    mid = (wave >= 8192 / 4) & (wave <= 8192)
    smooth = (8192 / wave[mid] - 1) / 3
    assert mid.any() and torch.allclose(f[mid], (1 - smooth) * plain[mid] / 8 + smooth * plain[mid], rtol=1e-14)
    f, scale = pkv.rope_inv_freq(64, 10000.0, scaling="yarn", factor=16.0, original_max_position=4096)
    assert math.isclose(scale, 0.1 * math.log(16.0) + 1.0)
    plain = 10000.0 ** (-p / 32)
    assert f[0] == plain[0] and math.isclose(float(f[-1]), float(plain[-1]) / 16, rel_tol=1e-12)
    assert bool((f <= plain * (1 + 1e-12)).all()) and bool((f >= plain / 16 * (1 - 1e-12)).all())
    assert bool((f[1:] < f[:-1]).all())
    for bad in (dict(rotary_dim=7), dict(rotary_dim=64, scaling="other"), dict(rotary_dim=64, factor=0.5),
                dict(rotary_dim=64, scaling="banded", low_freq_factor=4.0, high_freq_factor=1.0)):
        with pytest.raises(ValueError):
            pkv.rope_inv_freq(**bad)
