"""The prompt side of the paged cache (binding of the last part of include/pkv.h).

* ``qk_norm_rope_append`` takes a chunk's q, k and v from the projection: norm per head and
  rotation, q written for the attention, k and v into the pool;
* ``paged_prefill_attention`` attends a chunk of new tokens per sequence over the pool;
* ``paged_kv_gather`` reads cached positions back, dequantised;
* ``rope_inv_freq`` makes the rotation's frequencies, scaled for long contexts or not.
"""
from __future__ import annotations

import ctypes
import math
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


def _current(device: torch.device) -> None:
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")


def _beside(device: torch.device, **tensors: Optional[torch.Tensor]) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the cache on {device}")


def _empty(shape, dtype, device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A tensor whose memory is ordered with the call's stream, and safe to use from the current one."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _token_rows(name: str, t: torch.Tensor, heads: Optional[int], d: int) -> int:
    """Token stride of [T, heads, d] bf16 rows whose heads are contiguous."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if t.dim() != 3 or t.shape[2] != d or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [num_tokens, {'heads' if heads is None else heads}, {d}]")
    if t.shape[0] > 0 and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d)):
        raise ValueError(f"{name}'s heads must be contiguous (only the tokens may be strided)")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * d


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
      by factor from there up); rope_scale = 0.1 ln(factor) + 1.
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

        lo = max(0, math.floor(pair_turning(beta_fast)))
        hi = min(half - 1, math.ceil(pair_turning(beta_slow)))
        cut = ((p - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
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
    desc = _pkv._cache_desc(k_cache, v_cache, None, scales)
    device = k_cache.device
    _current(device)
    _beside(device, q=q, k=k, v=v, positions=positions, slot_mapping=slot_mapping, v_cache=v_cache, q_out=q_out,
            q_weight=q_weight, k_weight=k_weight, inv_freq=inv_freq, scales=scales)
    d, hkv = desc.head_dim, desc.num_kv_heads
    qs, ks, vs = _token_rows("q", q, None, d), _token_rows("k", k, hkv, d), _token_rows("v", v, hkv, d)
    T, hq = q.shape[0], q.shape[1]
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError("q, k and v must have the same number of tokens")
    if slot_mapping.dtype != torch.int64 or tuple(slot_mapping.shape) != (T,) or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 tensor [num_tokens]")
    if scales is not None and tuple(scales.shape) != (2, hkv):
        raise ValueError("scales must be [2, num_kv_heads]")
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None and (t.dtype != torch.bfloat16 or tuple(t.shape) != (d,) or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous bfloat16 tensor [head_dim]")
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float64 tensor [rotary_dim / 2]")
        if positions is None or positions.dtype != torch.int32 or tuple(positions.shape) != (T,) \
                or not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int32 tensor [num_tokens]")
        rot = 2 * inv_freq.shape[0]
    if q_out is None:
        q_out = _empty((T, hq, d), torch.bfloat16, device, stream)
    os = _token_rows("q_out", q_out, hq, d)
    if q_out.shape[0] != T:
        raise ValueError("q_out must have q's shape")
    a = RopeAppendDesc(q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
                       positions.data_ptr() if rot else None, slot_mapping.data_ptr(), T, hq, rot, int(interleaved),
                       rope_scale, inv_freq.data_ptr() if rot else None,
                       q_weight.data_ptr() if q_weight is not None else None,
                       k_weight.data_ptr() if k_weight is not None else None, eps, q_out.data_ptr(), os)
    _pkv._check(_pkv.lib.pkv_qk_norm_rope_append(ctypes.byref(desc), ctypes.byref(a), _pkv._stream(stream)))
    return q_out


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
    desc = _pkv._cache_desc(k_cache, v_cache, None, scales)
    device = k_cache.device
    _current(device)
    _beside(device, q=q, q_indptr=q_indptr, v_cache=v_cache, block_tables=block_tables, context_lens=context_lens,
            out=out, lse=lse, scales=scales, workspace=workspace)
    d, hkv = desc.head_dim, desc.num_kv_heads
    qs = _token_rows("q", q, None, d)
    T, hq = q.shape[0], q.shape[1]
    for name, t in (("q_indptr", q_indptr), ("block_tables", block_tables), ("context_lens", context_lens)):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous int32 tensor")
    B = context_lens.shape[0]
    if context_lens.dim() != 1 or tuple(q_indptr.shape) != (B + 1,):
        raise ValueError("context_lens must be [B] and q_indptr [B + 1]")
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be [B, max_blocks]")
    if scales is not None and tuple(scales.shape) != (2, hkv):
        raise ValueError("scales must be [2, num_kv_heads]")
    if max_context_len is None:
        max_context_len = block_tables.shape[1] * desc.block_size
    if out is None:
        out = _empty((T, hq, d), torch.bfloat16, device, stream)
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != (T, hq, d) or not out.is_contiguous():
        raise ValueError("out must be a contiguous bfloat16 tensor [T, Hq, D]")
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (T, hq) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor [T, Hq]")
    # a workspace of the call's own: calls on several streams and captured graphs share none
    need = prefill_workspace_size(B, T, hq, hkv, d, max_context_len) if B > 0 and T > 0 else 0
    ws_ptr, ws_bytes = None, 0
    if need > 0:
        ws = workspace if workspace is not None else _empty((need,), torch.uint8, device, stream)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _pkv._check(_pkv.lib.pkv_paged_prefill_attention(
        ctypes.byref(desc), q.data_ptr(), qs, q_indptr.data_ptr(), T, block_tables.data_ptr(), block_tables.shape[1],
        context_lens.data_ptr(), B, hq, max_context_len, int(causal), softmax_scale, out.data_ptr(),
        lse.data_ptr() if lse is not None else None, ws_ptr, ws_bytes, _pkv._stream(stream)))
    return out


def paged_kv_gather(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor, kv_indptr: torch.Tensor,
                    k_out: torch.Tensor, v_out: torch.Tensor, *, starts: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Read positions starts[b] .. (0 when None) of every sequence back into rows kv_indptr[b] ..
    kv_indptr[b + 1] of k_out and v_out ([rows, Hkv, D] bf16 or float32), dequantised.  Rows
    outside every range stay as they were."""
    desc = _pkv._cache_desc(k_cache, v_cache, None, scales)
    device = k_cache.device
    _current(device)
    _beside(device, v_cache=v_cache, block_tables=block_tables, kv_indptr=kv_indptr, k_out=k_out, v_out=v_out,
            starts=starts, scales=scales)
    for name, t in (("block_tables", block_tables), ("kv_indptr", kv_indptr), ("starts", starts)):
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous int32 tensor")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [B, max_blocks]")
    B = block_tables.shape[0]
    if tuple(kv_indptr.shape) != (B + 1,) or (starts is not None and tuple(starts.shape) != (B,)):
        raise ValueError("kv_indptr must be [B + 1] and starts [B]")
    if scales is not None and tuple(scales.shape) != (2, desc.num_kv_heads):
        raise ValueError("scales must be [2, num_kv_heads]")
    if k_out.dtype not in (torch.bfloat16, torch.float32) or k_out.dtype != v_out.dtype:
        raise TypeError("k_out and v_out must be both bfloat16 or both float32")
    rows = k_out.shape[0]
    if tuple(k_out.shape) != (rows, desc.num_kv_heads, desc.head_dim) or k_out.shape != v_out.shape \
            or not (k_out.is_contiguous() and v_out.is_contiguous()):
        raise ValueError("k_out and v_out must be contiguous [rows, num_kv_heads, head_dim]")
    _pkv._check(_pkv.lib.pkv_paged_kv_gather(
        ctypes.byref(desc), block_tables.data_ptr(), block_tables.shape[1], kv_indptr.data_ptr(),
        starts.data_ptr() if starts is not None else None, B, rows, k_out.data_ptr(), v_out.data_ptr(),
        _pkv.OUT_FP32 if k_out.dtype == torch.float32 else _pkv.OUT_BF16, _pkv._stream(stream)))
    return k_out, v_out
