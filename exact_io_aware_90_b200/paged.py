"""Torch wrappers of what stands around the attention: the norm and rotation of queries and keys (with its gradient), and
the paged key/value cache in 16 or 4 bits with the decode that reads it (``include/fa.h`` has the contracts).

A cache is two tensors, keys and values: [num_pages, Hk, page_size, d] of bfloat16 or float16, or uint8
[num_pages, Hk, page_size, 5·d/8] for 4 bits.  Nothing here synchronises; what the device finds out of range is reported by
``fa_check_device_status``.  Outputs and workspaces that a call allocates are allocated on the stream it runs on (``stream``,
else the current one).  Arguments are checked in ``_binding`` (csrc/binding.cpp).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import FA_BF16, FA_ERR_INVALID_ARG, FA_FP16, FA_OK, FAError, lib

try:
    from . import _binding
except ImportError as e:
    raise ImportError("the torch binding is missing or does not load: build it with "
                      "`python exact_io_aware_90_b200/build.py`. There is no fallback implementation.") from e

_binding.set_error_classes(FAError, torch.OutOfMemoryError)
_CODES = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16, None: -1}


def attention_rope_table(rows: int, rot_dim: int, base: float = 10000.0, device="cuda", stream=None):
    """(cos, sin), fp32 [rows, rot_dim / 2]: the angles position·base^(−2i / rot_dim), computed in 64 bits (fa_rope_table)."""
    if rows < 1 or rot_dim < 2:
        raise FAError(FA_ERR_INVALID_ARG, "fa_rope_table")
    with torch.cuda.device(device):
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(torch.cuda.ExternalStream(0 if stream == 1 else stream)):  # 1: the default stream too
            cos, sin = (torch.empty((rows, rot_dim // 2), dtype=torch.float32, device="cuda") for _ in range(2))
        st = lib.fa_rope_table(cos.data_ptr(), sin.data_ptr(), rows, rot_dim, float(base), stream)
    if st != FA_OK:
        raise FAError(st, "fa_rope_table")
    return cos, sin


def attention_qk_norm_rope(q, k, cos, sin, positions, wq=None, wk=None, eps: float = 1e-6, interleaved: bool = False,
                           sections=None, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): each head of q [T, Hq, d] and k [T, Hk, d] RMS-normed with wq, wk [d] (when given) and rotated by
    position; q and k may be slices of one projection's output (any token stride).  ``positions`` is int32 [T], or
    [axes, T] with ``sections`` (how many of the rot_dim/2 pairs go by each axis).  ``q_out=q`` works in place."""
    return _binding.qk_norm_rope(q, k, cos, sin, positions, sections, wq, wk, eps, interleaved, q_out, k_out, stream)


def attention_qk_norm_rope_backward(dq_out, dk_out, cos, sin, positions, q=None, k=None, wq=None, wk=None, eps: float = 1e-6,
                                    interleaved: bool = False, sections=None, dq=None, dk=None, dwq=None, dwk=None,
                                    workspace=None, stream=None):
    """(dq, dk, dwq, dwk) for the gradients dq_out, dk_out of ``attention_qk_norm_rope``'s outputs; with norm it needs the
    forward's q and k, and dwq, dwk are fp32 [d] (None without norm).  ``dq=dq_out`` works in place."""
    return _binding.qk_norm_rope_backward(dq_out, dk_out, cos, sin, positions, sections, q, k, wq, wk, eps, interleaved, dq, dk,
                                          dwq, dwk, workspace, stream)


def attention_cache_append(k, v, k_cache, v_cache, page_table, seqlens_k, cos=None, sin=None, positions=None, q=None, wq=None,
                           wk=None, eps: float = 1e-6, interleaved: bool = False, sections=None, cu_seqlens=None, q_out=None,
                           stream=None):
    """Appends k, v [T, Hk, d] to the paged cache, the keys normed (``wk``) and rotated (``cos``, ``sin``) on the way, and
    returns q normed and rotated the same way when it is given (else None).  ``seqlens_k`` holds the key counts after the
    append; ``cu_seqlens`` the sequences' rows (None: T/B each); ``positions`` those of the rotation (None: the positions in
    the cache)."""
    return _binding.cache_append(k, v, k_cache, v_cache, page_table, seqlens_k, cos, sin, positions, sections, q, wq, wk, eps,
                                 interleaved, cu_seqlens, q_out, stream)


def attention_cache_gather(k_cache, v_cache, page_table, cu_seqlens_k, total_keys: int, starts=None, dtype=None, k=None, v=None,
                           stream=None):
    """(k, v) [total_keys, Hk, d]: rows cu_seqlens_k[b] .. cu_seqlens_k[b+1] hold positions starts[b], starts[b] + 1, … of
    sequence b (starts None: 0; cu_seqlens_k None: total_keys/B rows each).  ``dtype`` is that of the rows of a 4-bit cache
    (None: k's, or bfloat16)."""
    if dtype not in _CODES:
        raise TypeError(f"unsupported dtype {dtype}: k and v are bfloat16 or float16")
    return _binding.cache_gather(k_cache, v_cache, page_table, cu_seqlens_k, total_keys, starts, _CODES[dtype], k, v, stream)


def attention_decode_paged(q, k_cache, v_cache, page_table, seqlens_k, max_seqlen_k: Optional[int] = None,
                           scale: Optional[float] = None, out=None, lse=None, workspace=None, stream=None):
    """O and LSE of the last tokens of each sequence over a paged cache: q [B, H, d] (one token each) or [B, Nq, H, d]; H a
    multiple of the cache's heads.  ``seqlens_k`` counts the keys, the new tokens' included; ``max_seqlen_k`` bounds them
    (None: the page table's capacity).  Query i of a sequence sees the keys up to position seqlens_k − Nq + i."""
    return _binding.decode_paged(q, k_cache, v_cache, page_table, seqlens_k, max_seqlen_k, scale, out, lse, workspace, stream)
