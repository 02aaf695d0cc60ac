"""Torch wrappers of what stands around the attention: the norm and rotation of queries and keys (with its gradient), and
the paged key/value cache in 16 or 4 bits with the decode that reads it (``include/fa.h`` has the contracts).

A cache is two tensors, keys and values: [num_pages, Hk, page_size, d] of bfloat16 or float16, or uint8
[num_pages, Hk, page_size, 5·d/8] for 4 bits.  Nothing here synchronises; what the device finds out of range is reported by
``fa_check_device_status``.  Outputs and workspaces that a call allocates are allocated on the stream it runs on.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch

from . import FA_BF16, FA_CACHE_16BIT, FA_CACHE_INT4, FA_ERR_INVALID_ARG, FA_FP16, FA_OK, FAError, lib

_CODES = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16}
_F32, _I32 = torch.float32, torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream  # what torch.cuda.current_stream wraps, at a thirtieth of its time

# The checks below are many per call and a call can take less time on the GPU than on the host, so each looks at a tensor's
# attributes once and in one expression.


def _code(dtype, name) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}: {name} must be bfloat16 or float16")
    return code


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _rows(t, name, dtype, device, T, d, heads=None):
    """(heads, token stride) of a [T, H, d] tensor whose heads and features are packed."""
    shape, stride = t.shape, t.stride()
    if (len(shape) != 3 or t.dtype != dtype or t.device != device or shape[0] != T or shape[2] != d or stride[2] != 1
            or (stride[1] != d and shape[1] != 1) or (heads is not None and heads != shape[1])):
        raise ValueError(f"{name} must be a {dtype} tensor [{T}, {'heads' if heads is None else heads}, {d}] on {device}, packed in "
                         f"heads and features (any token stride): got {t.dtype} {list(shape)} with strides {list(stride)} on {t.device}")
    return shape[1], stride[0] if T != 1 else shape[1] * d


def _flat(t, name, dtype, shape, device):
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {device}: got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _empty(like, shape, dtype, stream):
    """Memory of the stream the call runs on, so that the allocator reuses it in that stream's order."""
    if stream is None:
        return like.new_empty(shape) if like.dtype == dtype else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=like.device)):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _launch(where, fn, device, stream, *args):
    """fn(*args, stream) with the tensors' device current."""
    index = device.index
    if stream is None:
        stream = _raw_stream(index)
    if index == torch._C._cuda_getDevice():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream)
    if st != FA_OK:
        raise FAError(st, where)


@functools.lru_cache(maxsize=64)
def _sections_array(sections):
    return (ctypes.c_int * len(sections))(*sections)


def _rope(cos, sin, positions, sections, T, device):
    """(cos pointer, sin pointer, positions pointer, rot_dim, rows, axes, sections) of a rotation."""
    shape = cos.shape
    if len(shape) != 2:
        raise ValueError("cos and sin must be [rows, rot_dim / 2] tables")
    cp = _flat(cos, "cos", _F32, shape, device)
    sp = _flat(sin, "sin", _F32, shape, device)
    axes, arr = 1, None
    if sections is not None:
        if sum(sections) != shape[1]:
            raise ValueError("sections must add up to rot_dim / 2")
        axes, arr = len(sections), _sections_array(tuple(sections))
    pp = None
    if positions is not None:
        n = positions.shape
        if (positions.dtype != _I32 or positions.device != device or not positions.is_contiguous() or n[-1] != T
                or positions.numel() != axes * T):
            raise ValueError(f"positions must be a contiguous int32 tensor [{axes}, {T}] on {device}")
        pp = positions.data_ptr()
    return cp, sp, pp, 2 * shape[1], shape[0], axes, arr


def _weights(wq, wk, d, dtype, device):
    if wq is None and wk is None:
        return None, None
    if wk is None:
        raise ValueError("norm weights come in pairs: wk is missing")
    shape = (d,)
    return (None if wq is None else _flat(wq, "wq", dtype, shape, device)), _flat(wk, "wk", dtype, shape, device)


def attention_rope_table(rows: int, rot_dim: int, base: float = 10000.0, device="cuda", stream=None):
    """(cos, sin), fp32 [rows, rot_dim / 2]: the angles position·base^(−2i / rot_dim), computed in 64 bits (fa_rope_table)."""
    device = torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    if rows < 1 or rot_dim < 2:
        raise FAError(FA_ERR_INVALID_ARG, "fa_rope_table")
    like = torch.empty(0, dtype=_F32, device=device)
    cos, sin = (_empty(like, (rows, rot_dim // 2), _F32, stream) for _ in range(2))
    _launch("fa_rope_table", lib.fa_rope_table, device, stream, cos.data_ptr(), sin.data_ptr(), rows, rot_dim, float(base))
    return cos, sin


def attention_qk_norm_rope(q, k, cos, sin, positions, wq=None, wk=None, eps: float = 1e-6, interleaved: bool = False,
                           sections=None, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): each head of q [T, Hq, d] and k [T, Hk, d] RMS-normed with wq, wk [d] (when given) and rotated by
    position; q and k may be slices of one projection's output (any token stride).  ``positions`` is int32 [T], or
    [axes, T] with ``sections`` (how many of the rot_dim/2 pairs go by each axis).  ``q_out=q`` works in place."""
    dev, dtype = _cuda(q, "q"), q.dtype
    T, d = q.shape[0], q.shape[-1]
    Hq, sq = _rows(q, "q", dtype, dev, T, d)
    Hk, sk = _rows(k, "k", dtype, dev, T, d)
    if positions is None:
        raise ValueError("positions are required")
    if (wq is None) != (wk is None):
        raise ValueError("norm weights come in pairs")
    code = _code(dtype, "q")
    wqp, wkp = _weights(wq, wk, d, dtype, dev)
    cp, sp, pp, rot, rows, axes, arr = _rope(cos, sin, positions, sections, T, dev)
    if q_out is None:
        q_out, so = _empty(q, (T, Hq, d), dtype, stream), Hq * d
    else:
        so = _rows(q_out, "q_out", dtype, dev, T, d, Hq)[1]
    if k_out is None:
        k_out, to = _empty(q, (T, Hk, d), dtype, stream), Hk * d
    else:
        to = _rows(k_out, "k_out", dtype, dev, T, d, Hk)[1]
    _launch("fa_qk_norm_rope", lib.fa_qk_norm_rope, dev, stream, q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
            wqp, wkp, cp, sp, pp, T, Hq, Hk, d, sq, sk, so, to, rot, rows, axes, arr, int(interleaved), eps, code)
    return q_out, k_out


def attention_qk_norm_rope_backward(dq_out, dk_out, cos, sin, positions, q=None, k=None, wq=None, wk=None, eps: float = 1e-6,
                                    interleaved: bool = False, sections=None, dq=None, dk=None, dwq=None, dwk=None,
                                    workspace=None, stream=None):
    """(dq, dk, dwq, dwk) for the gradients dq_out, dk_out of ``attention_qk_norm_rope``'s outputs; with norm it needs the
    forward's q and k, and dwq, dwk are fp32 [d] (None without norm).  ``dq=dq_out`` works in place."""
    dev, dtype = _cuda(dq_out, "dq_out"), dq_out.dtype
    T, d = dq_out.shape[0], dq_out.shape[-1]
    Hq, gq = _rows(dq_out, "dq_out", dtype, dev, T, d)
    Hk, gk = _rows(dk_out, "dk_out", dtype, dev, T, d)
    if positions is None:
        raise ValueError("positions are required")
    if (wq is None) != (wk is None):
        raise ValueError("norm weights come in pairs")
    code = _code(dtype, "dq_out")
    cp, sp, pp, rot, rows, axes, arr = _rope(cos, sin, positions, sections, T, dev)
    wqp = wkp = qp = kp = dwqp = dwkp = ws = None
    sq = sk = ws_bytes = 0
    if wq is not None:
        if q is None or k is None:
            raise ValueError("q and k are needed for the norm's gradient")
        wqp, wkp = _weights(wq, wk, d, dtype, dev)
        sq, sk = _rows(q, "q", dtype, dev, T, d, Hq)[1], _rows(k, "k", dtype, dev, T, d, Hk)[1]
        qp, kp = q.data_ptr(), k.data_ptr()
        shape = (d,)
        if dwq is None:
            dwq = _empty(cos, shape, _F32, stream)
            dwqp = dwq.data_ptr()
        else:
            dwqp = _flat(dwq, "dwq", _F32, shape, dev)
        if dwk is None:
            dwk = _empty(cos, shape, _F32, stream)
            dwkp = dwk.data_ptr()
        else:
            dwkp = _flat(dwk, "dwk", _F32, shape, dev)
        if workspace is None:
            workspace = _empty(cos, _bwd_workspace(d) // 4, _F32, stream)
        elif workspace.device != dev:
            raise ValueError("workspace must be on the gradients' device")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        dwq = dwk = None
    if dq is None:
        dq, oq = _empty(dq_out, (T, Hq, d), dtype, stream), Hq * d
    else:
        oq = _rows(dq, "dq", dtype, dev, T, d, Hq)[1]
    if dk is None:
        dk, ok = _empty(dq_out, (T, Hk, d), dtype, stream), Hk * d
    else:
        ok = _rows(dk, "dk", dtype, dev, T, d, Hk)[1]
    _launch("fa_qk_norm_rope_bwd", lib.fa_qk_norm_rope_bwd, dev, stream, dq_out.data_ptr(), dk_out.data_ptr(), qp, kp, wqp, wkp,
            cp, sp, pp, dq.data_ptr(), dk.data_ptr(), dwqp, dwkp, T, Hq, Hk, d, gq, gk, sq, sk, oq, ok, rot, rows, axes, arr,
            int(interleaved), eps, code, ws, ws_bytes)
    return dq, dk, dwq, dwk


@functools.lru_cache(maxsize=8)
def _bwd_workspace(d):
    return max(lib.fa_qk_norm_rope_bwd_workspace_bytes(d), 256)


@functools.lru_cache(maxsize=256)
def _decode_workspace(B, Nq, H, Hk, Nk, d):
    return max(lib.fa_decode_paged_workspace_bytes(B, Nq, H, Hk, Nk, d), 256)


def _cache(k_cache, v_cache, page_table, device):
    """(d, Hk, page_size, num_pages, B, max_pages, format) of a cache and its page table."""
    shape, dtype = k_cache.shape, k_cache.dtype
    if (len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != dtype or k_cache.device != device or v_cache.device != device
            or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        raise ValueError(f"k_cache and v_cache must be alike, contiguous, [num_pages, Hk, page_size, row] on {device}")
    table = page_table.shape
    if len(table) != 2 or page_table.dtype != _I32 or page_table.device != device or not page_table.is_contiguous():
        raise ValueError(f"page_table must be a contiguous int32 tensor [B, max_pages] on {device}")
    pages, Hk, ps, row = shape
    if dtype == torch.uint8:
        if row % 5:
            raise ValueError("a 4-bit cache has rows of 5·d/8 bytes")
        return row // 5 * 8, Hk, ps, pages, table[0], table[1], FA_CACHE_INT4
    _code(dtype, "a 16-bit cache")
    return row, Hk, ps, pages, table[0], table[1], FA_CACHE_16BIT


def attention_cache_append(k, v, k_cache, v_cache, page_table, seqlens_k, cos=None, sin=None, positions=None, q=None, wq=None,
                           wk=None, eps: float = 1e-6, interleaved: bool = False, sections=None, cu_seqlens=None, q_out=None,
                           stream=None):
    """Appends k, v [T, Hk, d] to the paged cache, the keys normed (``wk``) and rotated (``cos``, ``sin``) on the way, and
    returns q normed and rotated the same way when it is given (else None).  ``seqlens_k`` holds the key counts after the
    append; ``cu_seqlens`` the sequences' rows (None: T/B each); ``positions`` those of the rotation (None: the positions in
    the cache)."""
    dev, dtype = _cuda(k, "k"), k.dtype
    T, d = k.shape[0], k.shape[-1]
    Hk, sk = _rows(k, "k", dtype, dev, T, d)
    sv = _rows(v, "v", dtype, dev, T, d, Hk)[1]
    code = _code(dtype, "k")
    cd, chk, ps, pages, B, most, fmt = _cache(k_cache, v_cache, page_table, dev)
    if cd != d or chk != Hk or (fmt == FA_CACHE_16BIT and k_cache.dtype != dtype):
        raise ValueError("the cache's heads, d and dtype must be those of k and v")
    lp = _flat(seqlens_k, "seqlens_k", _I32, (B,), dev)
    cu = None if cu_seqlens is None else _flat(cu_seqlens, "cu_seqlens", _I32, (B + 1,), dev)
    if q is None:
        if wq is not None:
            raise ValueError("wq without q")
    elif (wq is None) != (wk is None):
        raise ValueError("norm weights come in pairs")
    wqp, wkp = _weights(wq, wk, d, dtype, dev)
    if cos is not None and sin is not None:
        cp, sp, pp, rot, rows, axes, arr = _rope(cos, sin, positions, sections, T, dev)
    elif cos is not None or sin is not None:
        raise ValueError("cos and sin come in pairs")
    elif positions is not None or sections is not None:
        raise ValueError("positions and sections need cos and sin")
    else:
        cp, sp, pp, rot, rows, axes, arr = None, None, None, 0, 0, 1, None
    qp = op = None
    Hq = sq = so = 0
    if q is not None:
        Hq, sq = _rows(q, "q", dtype, dev, T, d)
        if q_out is None:
            q_out, so = _empty(q, (T, Hq, d), dtype, stream), Hq * d
        else:
            so = _rows(q_out, "q_out", dtype, dev, T, d, Hq)[1]
        qp, op = q.data_ptr(), q_out.data_ptr()
    _launch("fa_cache_append", lib.fa_cache_append, dev, stream, qp, k.data_ptr(), v.data_ptr(), op, k_cache.data_ptr(),
            v_cache.data_ptr(), wqp, wkp, cp, sp, pp, page_table.data_ptr(), lp, cu, B, T, Hq, Hk, d, sq, sk, sv, so, ps, pages,
            most, rot, rows, axes, arr, int(interleaved), eps, code, fmt)
    return q_out if q is not None else None


def attention_cache_gather(k_cache, v_cache, page_table, cu_seqlens_k, total_keys: int, starts=None, dtype=None, k=None, v=None,
                           stream=None):
    """(k, v) [total_keys, Hk, d]: rows cu_seqlens_k[b] .. cu_seqlens_k[b+1] hold positions starts[b], starts[b] + 1, … of
    sequence b (starts None: 0; cu_seqlens_k None: total_keys/B rows each).  ``dtype`` is that of the rows of a 4-bit cache
    (None: k's, or bfloat16)."""
    dev = _cuda(k_cache, "k_cache")
    d, Hk, ps, pages, B, most, fmt = _cache(k_cache, v_cache, page_table, dev)
    if fmt == FA_CACHE_16BIT:
        if dtype is not None and dtype != k_cache.dtype:
            raise ValueError("a 16-bit cache is read in its own dtype")
        dtype = k_cache.dtype
    elif dtype is None:
        dtype = k.dtype if k is not None else torch.bfloat16
    code = _code(dtype, "k")
    shape = (int(total_keys), Hk, d)
    if shape[0] < 1:
        raise FAError(FA_ERR_INVALID_ARG, "fa_cache_gather")
    cu = None if cu_seqlens_k is None else _flat(cu_seqlens_k, "cu_seqlens_k", _I32, (B + 1,), dev)
    sp = None if starts is None else _flat(starts, "starts", _I32, (B,), dev)
    if k is None:
        k = _empty(k_cache, shape, dtype, stream)
        kp = k.data_ptr()
    else:
        kp = _flat(k, "k", dtype, shape, dev)
    if v is None:
        v = _empty(k_cache, shape, dtype, stream)
        vp = v.data_ptr()
    else:
        vp = _flat(v, "v", dtype, shape, dev)
    _launch("fa_cache_gather", lib.fa_cache_gather, dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), kp, vp,
            page_table.data_ptr(), cu, sp, B, shape[0], Hk, d, ps, pages, most, code, fmt)
    return k, v


def attention_decode_paged(q, k_cache, v_cache, page_table, seqlens_k, max_seqlen_k: Optional[int] = None,
                           scale: Optional[float] = None, out=None, lse=None, workspace=None, stream=None):
    """O and LSE of the last tokens of each sequence over a paged cache: q [B, H, d] (one token each) or [B, Nq, H, d]; H a
    multiple of the cache's heads.  ``seqlens_k`` counts the keys, the new tokens' included; ``max_seqlen_k`` bounds them
    (None: the page table's capacity).  Query i of a sequence sees the keys up to position seqlens_k − Nq + i."""
    dev, dtype, shape = _cuda(q, "q"), q.dtype, q.shape
    if len(shape) == 4:
        Nq, H = shape[1], shape[2]
    elif len(shape) == 3:
        Nq, H = 1, shape[1]
    else:
        raise ValueError("q must be [B, H, d] or [B, Nq, H, d]")
    d, Hk, ps, pages, B, most, fmt = _cache(k_cache, v_cache, page_table, dev)
    if shape[0] != B or shape[-1] != d or (fmt == FA_CACHE_16BIT and k_cache.dtype != dtype) or not q.is_contiguous():
        raise ValueError("q must be contiguous, with the page table's batch and the cache's d and dtype")
    code = _code(dtype, "q")
    lp = _flat(seqlens_k, "seqlens_k", _I32, (B,), dev)
    Nk = most * ps if max_seqlen_k is None else int(max_seqlen_k)
    if out is None:
        out = _empty(q, shape, dtype, stream)
        op = out.data_ptr()
    else:
        op = _flat(out, "out", dtype, shape, dev)
    if lse is None:
        lse = _empty(q, shape[:-1], _F32, stream)
        ep = lse.data_ptr()
    else:
        ep = _flat(lse, "lse", _F32, shape[:-1], dev)
    if workspace is None:
        ws_bytes = _decode_workspace(B, Nq, H, Hk, Nk, d)
        workspace = _empty(seqlens_k, (ws_bytes + 3) // 4, _I32, stream)
    elif workspace.device != dev:
        raise ValueError("workspace must be on q's device")
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    _launch("fa_decode_paged", lib.fa_decode_paged, dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), op, ep,
            page_table.data_ptr(), lp, B, Nq, H, Hk, Nk, d, 1.0 / math.sqrt(d) if scale is None else scale, ps, pages, most, code, fmt,
            workspace.data_ptr(), ws_bytes)
    return out, lse
