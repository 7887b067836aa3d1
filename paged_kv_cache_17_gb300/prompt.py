"""The prompt side of the paged cache (binding of the last part of include/pkv.h).

* ``qk_norm_rope_append`` takes a chunk's q, k and v from the projection: norm per head and
  rotation, q written for the attention, k and v into the pool;
* ``paged_prefill_attention`` attends a chunk of new tokens per sequence over the pool;
* ``paged_kv_gather`` reads cached positions back, dequantised;
* ``rope_inv_freq`` makes the rotation's frequencies, scaled for long contexts or not.

Arguments are checked and marshalled by ``_pkv_prompt.so`` (``csrc/prompt_bind.cpp``); where it was not built,
the three calls raise ImportError.  Tensors must be on the current device.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
from typing import Optional, Tuple

import torch

import paged_kv_cache_17_gb300 as _pkv


class RopeAppendDesc(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("positions", ctypes.c_void_p), ("slot_mapping", ctypes.c_void_p), ("num_tokens", ctypes.c_int64),
                ("num_q_heads", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("rope_scale", ctypes.c_float), ("inv_freq", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float), ("q_out", ctypes.c_void_p),
                ("q_out_stride", ctypes.c_int64)]


def bind(lib: ctypes.CDLL) -> None:
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    cache = ctypes.POINTER(_pkv.CacheDesc)
    lib.pkv_qk_norm_rope_append.restype = ctypes.c_int
    lib.pkv_qk_norm_rope_append.argtypes = [cache, ctypes.POINTER(RopeAppendDesc), P]
    lib.pkv_prefill_workspace_size.restype = sz
    lib.pkv_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.pkv_paged_prefill_attention.restype = ctypes.c_int
    lib.pkv_paged_prefill_attention.argtypes = [cache, P, i64, P, i32, P, i32, P, i32, i32, i32, i32, ctypes.c_float,
                                                P, P, P, sz, P]
    lib.pkv_paged_kv_gather.restype = ctypes.c_int
    lib.pkv_paged_kv_gather.argtypes = [cache, P, i32, P, P, i32, i64, P, P, ctypes.c_int, P]


bind(_pkv.lib)


class _Missing:
    """Stands in for the module of the marshalled calls where it cannot be loaded: they raise, what does not
    need it works."""

    def __init__(self, why: str):
        self._why = why

    def __getattr__(self, name: str):
        raise ImportError(self._why)


def _marshal():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "_pkv_prompt.so")
    if not os.path.exists(path):
        return _Missing(f"_pkv_prompt.so is not built ({path}); run python -m paged_kv_cache_17_gb300._build")
    spec = importlib.util.spec_from_file_location("_pkv_prompt", path)
    try:
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    except ImportError as e:  # built against another torch
        return _Missing(f"{path} cannot be loaded ({e}); run python -m paged_kv_cache_17_gb300._build")
    return mod


_bind = _marshal()


def _run(call, stream: Optional[torch.cuda.Stream], *args):
    """The call on the current stream, or on the one given: the memory it takes is then that stream's,
    and an output it made may be used on the current one."""
    if stream is None:
        r = call(*args)
    else:
        now = torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            r = call(*args)
        if r.__class__ is not int and not any(r is a for a in args):
            r.record_stream(now)
    if r.__class__ is int:
        _pkv._check(r)
    return r


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, *, scaling: Optional[str] = None, factor: float = 1.0,
                  original_max_position: int = 8192, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
                  beta_fast: float = 32.0, beta_slow: float = 1.0,
                  device: Optional[torch.device] = None) -> Tuple[torch.Tensor, float]:
    """(inv_freq [rotary_dim / 2] float64 in radians per position, rope_scale) for
    qk_norm_rope_append.  inv_freq[p] = base^(-2p / rotary_dim), then by ``scaling``:

    * None: as it is;
    * "linear": divided by factor (positions interpolated);
    * "ntk": base raised by factor^(R / (R - 2)), R = rotary_dim: the fastest pair keeps its
      frequency, the slowest is divided by factor;
    * "banded": pairs with a wavelength above original_max_position / low_freq_factor are divided
      by factor, those below original_max_position / high_freq_factor kept, and between the two
      blended linearly in original_max_position / wavelength;
    * "yarn": blended linearly in the pair index between the pair that turns beta_fast times over
      original_max_position (kept from there down) and the one that turns beta_slow times (divided
      by factor from there up), the former's index rounded down, at least 0, the latter's up, at most
      R - 1; rope_scale = 0.1 ln(factor) + 1.
    """
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be positive and even")
    if not (factor >= 1.0 and base > 1.0 and original_max_position > 0):
        raise ValueError("factor must be >= 1, base > 1 and original_max_position positive")
    if scaling == "ntk":
        if rotary_dim <= 2:
            raise ValueError("ntk scaling needs rotary_dim > 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    half = rotary_dim // 2
    p = torch.arange(half, dtype=torch.float64)
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -p / half)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "banded":
        if not 0 < low_freq_factor < high_freq_factor:
            raise ValueError("low_freq_factor must be positive and below high_freq_factor")
        turns = original_max_position * f / (2 * math.pi)
        keep = ((turns - low_freq_factor) / (high_freq_factor - low_freq_factor)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    elif scaling == "yarn":
        if not 0 < beta_slow < beta_fast:
            raise ValueError("beta_slow must be positive and below beta_fast")

        def pair_turning(times):  # index (not whole) of the pair that turns so often
            return half * math.log(original_max_position / (2 * math.pi * times)) / math.log(base)

        # (the end may lie behind the last pair: the ramp then runs on to it)
        lo = max(0, math.floor(pair_turning(beta_fast)))
        hi = min(rotary_dim - 1, math.ceil(pair_turning(beta_slow)))
        cut = ((p - lo) / max(hi - lo, 1e-3)).clamp(0, 1) if hi >= 0 else torch.ones_like(p)
        f = f * ((1 - cut) + cut / factor)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device) if device is not None else f, scale


def qk_norm_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: Optional[torch.Tensor],
                        slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        q_out: Optional[torch.Tensor] = None, *, q_weight: Optional[torch.Tensor] = None,
                        k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False, rope_scale: float = 1.0,
                        scales: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Norm (q_weight, k_weight: [D] bf16, None for no norm) and rotate (inv_freq: [R / 2] float64,
    None for no rotation; positions [T] int32) the heads of q [T, Hq, D] and k [T, Hkv, D], write
    q to q_out (allocated when None; may be q) and k, v into the pools at slot_mapping ([T] int64;
    negative: not written).  bf16; the token dimension of q, k, v and q_out may be strided."""
    return _run(_bind.append, stream, q, k, v, positions, slot_mapping, k_cache, v_cache, q_out, q_weight, k_weight, eps,
                inv_freq, interleaved, rope_scale, scales)


def prefill_workspace_size(batch: int, total_q: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                           max_context_len: int) -> int:
    return int(_pkv.lib.pkv_prefill_workspace_size(batch, total_q, num_q_heads, num_kv_heads, head_dim,
                                                   max_context_len))


def paged_prefill_attention(q: torch.Tensor, q_indptr: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, context_lens: torch.Tensor, softmax_scale: float,
                            out: Optional[torch.Tensor] = None, *, causal: bool = True,
                            lse: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                            max_context_len: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of chunks of new tokens over the paged cache that already holds them.

    q: [T, Hq, D] bf16 (tokens may be strided), the rows of sequence b at q_indptr[b] ..
    q_indptr[b + 1] (int32 [B + 1]).  block_tables [B, max_blocks] and context_lens [B] int32;
    context_lens counts the chunk when causal.  Row i of n of a sequence with context c sees the
    keys up to its position c - n + i (causal), or all c.  out: [T, Hq, D] bf16 (allocated when
    None); lse: float32 [T, Hq], written when given.  Rows behind the last sequence stay as they
    were.  max_context_len defaults to the table capacity."""
    return _run(_bind.prefill, stream, q, q_indptr, k_cache, v_cache, block_tables, context_lens, softmax_scale, out,
                causal, lse, scales, max_context_len, workspace)


def paged_kv_gather(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor, kv_indptr: torch.Tensor,
                    k_out: torch.Tensor, v_out: torch.Tensor, *, starts: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Read positions starts[b] .. (0 when None) of every sequence back into rows kv_indptr[b] ..
    kv_indptr[b + 1] of k_out and v_out ([rows, Hkv, D] bf16 or float32), dequantised.  Rows
    outside every range stay as they were."""
    _run(_bind.gather, stream, k_cache, v_cache, block_tables, kv_indptr, k_out, v_out, starts, scales)
    return k_out, v_out
