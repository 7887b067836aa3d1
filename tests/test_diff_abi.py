"""Differential attention without a GPU: refusals by the C ABI before any CUDA call, and by the binding."""
import ctypes
import math

import pytest
import torch

from test_prompt_abi import desc, last

NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_17_gb300 as m

    return m


def diff(**kw):
    from paged_kv_cache_17_gb300.diff import DiffDesc

    a = dict(lambda_=0xa0000, lambda_stride=0, norm_weight=None, eps=1e-5, out_scale=1.0)
    a.update(kw)
    return DiffDesc(**a)


def prefill(pkv, d, f=None, q=0x600000, stride=512, indptr=0x50000, T=10, tables=0x80000, blocks=7, lens=0x90000, B=4, hq=8,
            max_len=100, causal=1, scale=0.125, out=0x700000):
    f = diff() if f is None else f
    return pkv.lib.pkv_paged_diff_prefill_attention(ctypes.byref(d), q, stride, indptr, T, tables, blocks, lens, B, hq,
                                                    max_len, causal, scale, ctypes.byref(f) if f else None, out, None, 0, None)


def step(pkv, d, f=None, q=0x600000, tables=0x80000, blocks=7, lens=0x90000, B=4, hq=8, max_len=100, scale=0.125,
         out=0x700000, dt=0):
    f = diff() if f is None else f
    return pkv.lib.pkv_paged_diff_decode_attention(ctypes.byref(d), q, tables, blocks, lens, B, hq, max_len, scale,
                                                   ctypes.byref(f) if f else None, out, dt, None, 0, None)


def cascade(pkv, d, f=None, q=0x600000, tables=0x80000, blocks=7, lens=0x90000, B=4, hq=8, max_len=100, scale=0.125,
            out=0x700000, dt=0, **kw):
    f = diff() if f is None else f
    x = dict(prefix_tables=0xb0000, max_prefix_blocks=4, prefix_lens=0xc0000, num_prefixes=1, member_indptr=0xd0000,
             member_seqs=0xe0000, max_members=2, max_prefix_len=64, seq_prefix=0xf0000)
    x.update(kw)
    px = pkv.PrefixDesc(**x)
    return pkv.lib.pkv_cascade_diff_decode_attention(ctypes.byref(d), q, ctypes.byref(px), tables, blocks, lens, B, hq,
                                                     max_len, scale, ctypes.byref(f) if f else None, out, dt, None, 0, None)


CALLS = [prefill, step, cascade]


@pytest.mark.parametrize("call", CALLS)
def test_refusals_of_every_form(pkv, call):
    bad, unsup = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED
    d = desc(pkv)
    assert call(pkv, d, B=0) == pkv.PKV_OK  # nothing to do, no CUDA call
    assert call(pkv, desc(pkv, head_dim=128)) == unsup and "head_dim" in last(pkv)
    assert call(pkv, desc(pkv, block_size=32)) == unsup
    assert call(pkv, desc(pkv, kv_dtype=1)) == bad and "scales" in last(pkv)
    assert call(pkv, desc(pkv, num_kv_heads=1), hq=8) == bad and "pairs" in last(pkv)
    assert call(pkv, desc(pkv, num_kv_heads=3), hq=3) == bad and "pairs" in last(pkv)
    assert call(pkv, d, hq=6) == unsup and "group" in last(pkv)
    assert call(pkv, d, hq=5) == bad and call(pkv, d, hq=0) == bad
    assert call(pkv, d, hq=32) == unsup  # a query group of 16
    assert call(pkv, d, B=-1) == bad and call(pkv, d, B=70000) == bad
    for name in ("q", "tables", "lens", "out"):
        assert call(pkv, d, **{name: None}) == bad
    assert call(pkv, d, q=0x600008) == bad and call(pkv, d, out=0x700008) == bad
    assert call(pkv, d, lens=0x90002) == bad and call(pkv, d, tables=0x80001) == bad
    assert call(pkv, d, max_len=113) == bad and "max_blocks_per_seq" in last(pkv)
    assert call(pkv, d, max_len=-1) == bad and call(pkv, d, blocks=0, max_len=0) == bad
    assert call(pkv, d, max_len=(1 << 30) + 1, blocks=1 << 27) == unsup
    for scale in (NAN, INF, 2e38):
        assert call(pkv, d, scale=scale) == bad and "softmax_scale" in last(pkv)
    assert call(pkv, d, f=False) == bad and "descriptor" in last(pkv)
    for kw in (dict(lambda_=None), dict(lambda_=0xa0002), dict(lambda_stride=3), dict(lambda_stride=-4),
               dict(norm_weight=0x100008), dict(norm_weight=0x100000, eps=-1.0), dict(norm_weight=0x100000, eps=NAN),
               dict(out_scale=INF)):
        assert call(pkv, d, f=diff(**kw)) == bad, kw
    row = 8 * 64 * 2
    for out in (0x600000, 0x600000 + 3 * row, 0x600000 - row, 0x600010):
        assert call(pkv, d, out=out) == bad and "overlaps" in last(pkv)


def test_refusals_of_the_chunk(pkv):
    bad, d = pkv.PKV_ERR_INVALID_ARG, desc(pkv)
    assert prefill(pkv, d, T=0) == pkv.PKV_OK and prefill(pkv, d, T=-1) == bad
    assert prefill(pkv, d, stride=504) == bad and "stride" in last(pkv)
    assert prefill(pkv, d, stride=513) == bad
    assert prefill(pkv, d, indptr=None) == bad and prefill(pkv, d, indptr=0x50001) == bad
    assert prefill(pkv, d, causal=2) == bad
    assert pkv.lib.pkv_diff_prefill_workspace_size(4, 10, 8, 2, 128, 100) == 0 and "head_dim" in last(pkv)
    assert pkv.lib.pkv_diff_prefill_workspace_size(4, 10, 6, 2, 64, 100) == 0 and "group" in last(pkv)


def test_refusals_of_one_token(pkv):
    bad, d = pkv.PKV_ERR_INVALID_ARG, desc(pkv)
    for call in (step, cascade):
        assert call(pkv, d, dt=2) == bad
        # fp32 rows are twice as long
        assert call(pkv, d, dt=1, out=0x600000 - 5 * 1024) == bad and "overlaps" in last(pkv)
    assert pkv.lib.pkv_diff_decode_workspace_size(4, 8, 3, 64, 100) == 0
    assert pkv.lib.pkv_cascade_diff_workspace_size(4, 8, 2, 64, 100, 1, -1, 64) == 0 and "prefix" in last(pkv)


def test_refusals_of_prefixes(pkv):
    bad, d = pkv.PKV_ERR_INVALID_ARG, desc(pkv)
    assert pkv.lib.pkv_cascade_diff_decode_attention(ctypes.byref(d), 0x600000, None, 0x80000, 7, 0x90000, 4, 8, 100, 0.125,
                                                     ctypes.byref(diff()), 0x700000, 0, None, 0, None) == bad
    for name in ("num_prefixes", "max_members", "max_prefix_len", "max_prefix_blocks"):
        assert cascade(pkv, d, **{name: -1}) == bad
    for name in ("prefix_tables", "prefix_lens", "member_indptr", "member_seqs", "seq_prefix"):
        assert cascade(pkv, d, **{name: None}) == bad
        assert cascade(pkv, d, **{name: 0xb0001}) == bad and "aligned" in last(pkv)
    assert cascade(pkv, d, max_prefix_len=60) == bad and "multiple" in last(pkv)
    assert cascade(pkv, d, max_prefix_len=80) == bad and "max_prefix_blocks" in last(pkv)


def test_binding_refuses_tensors_that_are_not_on_a_gpu(pkv):
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((1, 8, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((1, 4), dtype=torch.int32)
    lam = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.paged_diff_prefill_attention(q, i, k, k.clone(), t, i[:1], 0.1, lam)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.paged_diff_decode_attention(q, k, k.clone(), t, i[:1], 0.1, lam)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.cascade_diff_decode_attention(q, k, k.clone(), t, i[:1], i, i[:1], i[:1], t, i[:1], 0.1, lam, max_members=1)
    with pytest.raises(TypeError):
        pkv.paged_diff_decode_attention(q, None, k, t, i[:1], 0.1, lam)
