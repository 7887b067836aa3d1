"""Differential attention over the paged cache (binding of the part of include/pkv.h on it).

Heads of 64 elements come in pairs: output head p has the queries 2p and 2p + 1, the keys of kv heads 2n and 2n + 1
and the values of both side by side (n the kv pair of p's group), and is the difference of the two softmax maps,
the second times ``lam``, over those values; then, with ``norm_weight``, the RMS norm of its 128 elements, and
``out_scale``.

* ``paged_diff_prefill_attention`` attends a chunk of new tokens per sequence;
* ``paged_diff_decode_attention`` attends one token per sequence;
* ``cascade_diff_decode_attention`` attends one token per sequence where sequences share prefixes, each prefix once;
* ``diff_lambda`` makes ``lam`` from the vectors that a model learns.

The pool is an ordinary one, filled by ``paged_kv_append`` or ``qk_norm_rope_append``.  Arguments are checked and
marshalled by ``_pkv_prompt.so``; tensors must be on the current device.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

import paged_kv_cache_17_gb300 as _pkv

from .prompt import _bind, _run


class DiffDesc(ctypes.Structure):
    _fields_ = [("lambda_", ctypes.c_void_p), ("lambda_stride", ctypes.c_int64), ("norm_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("out_scale", ctypes.c_float)]


def bind(lib: ctypes.CDLL) -> None:
    P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    cache, desc = ctypes.POINTER(_pkv.CacheDesc), ctypes.POINTER(DiffDesc)
    lib.pkv_diff_prefill_workspace_size.restype = sz
    lib.pkv_diff_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.pkv_paged_diff_prefill_attention.restype = ctypes.c_int
    lib.pkv_paged_diff_prefill_attention.argtypes = [cache, P, i64, P, i32, P, i32, P, i32, i32, i32, i32, f32, desc, P, P,
                                                     sz, P]
    lib.pkv_diff_decode_workspace_size.restype = sz
    lib.pkv_diff_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.pkv_paged_diff_decode_attention.restype = ctypes.c_int
    lib.pkv_paged_diff_decode_attention.argtypes = [cache, P, P, i32, P, i32, i32, i32, f32, desc, P, ctypes.c_int, P, sz, P]
    lib.pkv_cascade_diff_workspace_size.restype = sz
    lib.pkv_cascade_diff_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32]
    lib.pkv_cascade_diff_decode_attention.restype = ctypes.c_int
    lib.pkv_cascade_diff_decode_attention.argtypes = [cache, P, ctypes.POINTER(_pkv.PrefixDesc), P, i32, P, i32, i32, i32,
                                                      f32, desc, P, ctypes.c_int, P, sz, P]


bind(_pkv.lib)


def diff_lambda(q1: torch.Tensor, k1: torch.Tensor, q2: torch.Tensor, k2: torch.Tensor, init: float) -> torch.Tensor:
    """exp(q1 . k1) - exp(q2 . k2) + init over the last dimension, float32 from sums in float64: [heads] from
    learned vectors [heads, d], or a value from [d], to be expanded to [heads]."""
    a, b = ((x.double() * y.double()).sum(-1).exp() for x, y in ((q1, k1), (q2, k2)))
    return (a - b + init).float()


def diff_prefill_workspace_size(batch: int, total_q: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                max_context_len: int) -> int:
    return int(_pkv.lib.pkv_diff_prefill_workspace_size(batch, total_q, num_q_heads, num_kv_heads, head_dim,
                                                        max_context_len))


def diff_decode_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                               max_context_len: int) -> int:
    return int(_pkv.lib.pkv_diff_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_context_len))


def cascade_diff_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_context_len: int,
                                num_prefixes: int, max_members: int, max_prefix_len: int) -> int:
    return int(_pkv.lib.pkv_cascade_diff_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                                        num_prefixes, max_members, max_prefix_len))


def paged_diff_prefill_attention(q: torch.Tensor, q_indptr: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                 block_tables: torch.Tensor, context_lens: torch.Tensor, softmax_scale: float,
                                 lam: torch.Tensor, out: Optional[torch.Tensor] = None, *,
                                 norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-5, out_scale: float = 1.0,
                                 causal: bool = True, scales: Optional[torch.Tensor] = None,
                                 max_context_len: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Differential attention of chunks of new tokens over the paged cache that already holds them: q [T, Hq, 64]
    bf16 and the tables as for paged_prefill_attention; lam float32 [Hq / 2] or [T, Hq / 2] (tokens may be
    strided); norm_weight [128] bf16, None for no norm.  out: [T, Hq / 2, 128] bf16 (allocated when None); rows
    behind the last sequence stay as they were."""
    return _run(_bind.diff_prefill, stream, q, q_indptr, k_cache, v_cache, block_tables, context_lens, softmax_scale, lam,
                out, norm_weight, eps, out_scale, causal, scales, max_context_len, workspace)


def paged_diff_decode_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                block_tables: torch.Tensor, context_lens: torch.Tensor, softmax_scale: float,
                                lam: torch.Tensor, out: Optional[torch.Tensor] = None, *,
                                norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-5, out_scale: float = 1.0,
                                scales: Optional[torch.Tensor] = None, max_context_len: Optional[int] = None,
                                workspace: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Differential attention of one token per sequence: q [B, Hq, 64] bf16, contiguous, and the tables as for
    paged_decode_attention; lam float32 [Hq / 2] or [B, Hq / 2]; norm_weight [128] bf16, None for no norm.  out:
    [B, Hq / 2, 128] bf16 or float32 (allocated as bf16 when None)."""
    return _run(_bind.diff_decode, stream, q, k_cache, v_cache, block_tables, context_lens, softmax_scale, lam, out,
                norm_weight, eps, out_scale, scales, max_context_len, workspace)


def cascade_diff_decode_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  prefix_tables: torch.Tensor, prefix_lens: torch.Tensor, member_indptr: torch.Tensor,
                                  member_seqs: torch.Tensor, seq_prefix: torch.Tensor, block_tables: torch.Tensor,
                                  context_lens: torch.Tensor, softmax_scale: float, lam: torch.Tensor,
                                  out: Optional[torch.Tensor] = None, *, max_members: int,
                                  norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-5, out_scale: float = 1.0,
                                  max_prefix_len: Optional[int] = None, max_context_len: Optional[int] = None,
                                  scales: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Differential attention of one token per sequence where sequences share prefixes: the prefixes as for
    cascade_decode_attention, everything else as for paged_diff_decode_attention; block_tables and context_lens hold
    each sequence's blocks after its prefix."""
    return _run(_bind.diff_cascade, stream, q, k_cache, v_cache, prefix_tables, prefix_lens, member_indptr, member_seqs,
                seq_prefix, block_tables, context_lens, softmax_scale, lam, out, norm_weight, eps, out_scale, max_members,
                max_prefix_len, max_context_len, scales, workspace)
