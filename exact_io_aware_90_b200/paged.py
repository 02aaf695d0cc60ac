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

from . import FA_BF16, FA_CACHE_16BIT, FA_CACHE_INT4, FA_FP16, FA_OK, FAError, lib

_CODES = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16}


def _code(t, name) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}: {name} must be bfloat16 or float16")
    return code


def _rows(t, name, like=None, heads=None):
    """Token stride of a CUDA [T, H, d] tensor whose heads and features are packed."""
    if t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [T, heads, d]")
    T, H, d = t.shape
    if like is not None and (t.dtype != like.dtype or t.device != like.device or T != like.shape[0] or d != like.shape[2]):
        raise ValueError(f"{name} must have the dtype, device, token count and d of the other rows")
    if heads is not None and H != heads:
        raise ValueError(f"{name} must have {heads} heads")
    s = t.stride()
    if s[2] != 1 or (H > 1 and s[1] != d):
        raise ValueError(f"{name} must be packed in heads and features (any token stride)")
    return s[0] if T > 1 else H * d


def _flat(t, name, dtype, shape, device):
    if not t.is_cuda or not t.is_contiguous() or t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device:
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor {list(shape)} on {device}")
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """Memory of the stream the call runs on, so that the allocator reuses it in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _launch(where, fn, device, stream, *args):
    """fn(*args, stream) with the tensors' device current."""
    if stream is None:
        stream = torch.cuda.current_stream(device).cuda_stream
    if device.index is None or device.index == torch.cuda.current_device():
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
    if cos.dim() != 2:
        raise ValueError("cos and sin must be [rows, rot_dim / 2] tables")
    cp = _flat(cos, "cos", torch.float32, cos.shape, device)
    sp = _flat(sin, "sin", torch.float32, cos.shape, device)
    axes = 1 if sections is None else len(sections)
    pp = None
    if positions is not None:
        n = positions.numel()
        if (not positions.is_cuda or positions.dtype != torch.int32 or not positions.is_contiguous() or positions.device != device
                or n != axes * T or positions.shape[-1] != T):
            raise ValueError(f"positions must be a contiguous CUDA int32 tensor [{axes}, {T}] on {device}")
        pp = positions.data_ptr()
    arr = None if axes == 1 and (sections is None or sections[0] == cos.shape[1]) else _sections_array(tuple(sections))
    if sections is not None and sum(sections) != cos.shape[1]:
        raise ValueError("sections must add up to rot_dim / 2")
    return cp, sp, pp, 2 * cos.shape[1], cos.shape[0], axes, arr


def _weights(wq, wk, d, dtype, device):
    if wq is None and wk is None:
        return None, None
    if wk is None:
        raise ValueError("norm weights come in pairs: wk is missing")
    return (None if wq is None else _flat(wq, "wq", dtype, (d,), device)), _flat(wk, "wk", dtype, (d,), device)


def attention_rope_table(rows: int, rot_dim: int, base: float = 10000.0, device="cuda", stream=None):
    """(cos, sin), fp32 [rows, rot_dim / 2]: the angles position·base^(−2i / rot_dim), computed in 64 bits (fa_rope_table)."""
    device = torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    if rows < 1 or rot_dim < 2:
        raise FAError(1, "fa_rope_table")
    cos = _empty((rows, rot_dim // 2), torch.float32, device, stream)
    sin = _empty((rows, rot_dim // 2), torch.float32, device, stream)
    _launch("fa_rope_table", lib.fa_rope_table, device, stream, cos.data_ptr(), sin.data_ptr(), rows, rot_dim, float(base))
    return cos, sin


def attention_qk_norm_rope(q, k, cos, sin, positions, wq=None, wk=None, eps: float = 1e-6, interleaved: bool = False,
                           sections=None, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): each head of q [T, Hq, d] and k [T, Hk, d] RMS-normed with wq, wk [d] (when given) and rotated by
    position; q and k may be slices of one projection's output (any token stride).  ``positions`` is int32 [T], or
    [axes, T] with ``sections`` (how many of the rot_dim/2 pairs go by each axis).  ``q_out=q`` works in place."""
    sq, sk = _rows(q, "q"), _rows(k, "k", q)
    T, Hq, d = q.shape
    Hk, dev = k.shape[1], q.device
    if positions is None:
        raise ValueError("positions are required")
    w = _weights(wq, wk, d, q.dtype, dev)
    if (wq is None) != (wk is None):
        raise ValueError("norm weights come in pairs")
    cp, sp, pp, rot, rows, axes, arr = _rope(cos, sin, positions, sections, T, dev)
    code = _code(q, "q")
    if q_out is None:
        q_out = _empty((T, Hq, d), q.dtype, dev, stream)
        so = Hq * d
    else:
        so = _rows(q_out, "q_out", q, Hq)
    if k_out is None:
        k_out = _empty((T, Hk, d), q.dtype, dev, stream)
        to = Hk * d
    else:
        to = _rows(k_out, "k_out", q, Hk)
    _launch("fa_qk_norm_rope", lib.fa_qk_norm_rope, dev, stream, q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
            w[0], w[1], cp, sp, pp, T, Hq, Hk, d, sq, sk, so, to, rot, rows, axes, arr, int(interleaved), float(eps), code)
    return q_out, k_out


def attention_qk_norm_rope_backward(dq_out, dk_out, cos, sin, positions, q=None, k=None, wq=None, wk=None, eps: float = 1e-6,
                                    interleaved: bool = False, sections=None, dq=None, dk=None, dwq=None, dwk=None,
                                    workspace=None, stream=None):
    """(dq, dk, dwq, dwk) for the gradients dq_out, dk_out of ``attention_qk_norm_rope``'s outputs; with norm it needs the
    forward's q and k, and dwq, dwk are fp32 [d] (None without norm).  ``dq=dq_out`` works in place."""
    gq, gk = _rows(dq_out, "dq_out"), _rows(dk_out, "dk_out", dq_out)
    T, Hq, d = dq_out.shape
    Hk, dev = dk_out.shape[1], dq_out.device
    if positions is None:
        raise ValueError("positions are required")
    w = _weights(wq, wk, d, dq_out.dtype, dev)
    if (wq is None) != (wk is None):
        raise ValueError("norm weights come in pairs")
    cp, sp, pp, rot, rows, axes, arr = _rope(cos, sin, positions, sections, T, dev)
    code = _code(dq_out, "dq_out")
    qp = kp = wqp = wkp = ws = None
    sq = sk = ws_bytes = 0
    if wq is not None:
        if q is None or k is None:
            raise ValueError("q and k are needed for the norm's gradient")
        sq, sk = _rows(q, "q", dq_out, Hq), _rows(k, "k", dq_out, Hk)
        qp, kp = q.data_ptr(), k.data_ptr()
        dwq = _empty((d,), torch.float32, dev, stream) if dwq is None else dwq
        dwk = _empty((d,), torch.float32, dev, stream) if dwk is None else dwk
        wqp, wkp = _flat(dwq, "dwq", torch.float32, (d,), dev), _flat(dwk, "dwk", torch.float32, (d,), dev)
        ws_bytes = lib.fa_qk_norm_rope_bwd_workspace_bytes(d)
        if workspace is None:
            workspace = _empty((max(ws_bytes, 1),), torch.uint8, dev, stream)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        dwq = dwk = None
    if dq is None:
        dq = _empty((T, Hq, d), dq_out.dtype, dev, stream)
    if dk is None:
        dk = _empty((T, Hk, d), dq_out.dtype, dev, stream)
    oq, ok = _rows(dq, "dq", dq_out, Hq), _rows(dk, "dk", dq_out, Hk)
    _launch("fa_qk_norm_rope_bwd", lib.fa_qk_norm_rope_bwd, dev, stream, dq_out.data_ptr(), dk_out.data_ptr(), qp, kp, w[0], w[1],
            cp, sp, pp, dq.data_ptr(), dk.data_ptr(), wqp, wkp, T, Hq, Hk, d, gq, gk, sq, sk, oq, ok, rot, rows, axes, arr,
            int(interleaved), float(eps), code, ws, ws_bytes)
    return dq, dk, dwq, dwk


def _cache(k_cache, v_cache, page_table):
    """(d, Hk, page_size, num_pages, B, max_pages, format) of a cache and its page table."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype or k_cache.device != v_cache.device:
        raise ValueError("k_cache and v_cache must be alike, [num_pages, Hk, page_size, row]")
    if not k_cache.is_cuda or not k_cache.is_contiguous() or not v_cache.is_contiguous():
        raise ValueError("k_cache and v_cache must be contiguous CUDA tensors")
    if (page_table.dim() != 2 or page_table.dtype != torch.int32 or not page_table.is_contiguous()
            or page_table.device != k_cache.device):
        raise ValueError("page_table must be a contiguous int32 tensor [B, max_pages] on the cache's device")
    pages, Hk, ps, row = k_cache.shape
    B, most = page_table.shape
    if k_cache.dtype == torch.uint8:
        if row % 5:
            raise ValueError("a 4-bit cache has rows of 5·d/8 bytes")
        return row // 5 * 8, Hk, ps, pages, B, most, FA_CACHE_INT4
    _code(k_cache, "a 16-bit cache")
    return row, Hk, ps, pages, B, most, FA_CACHE_16BIT


def _lens(t, name, n, device):
    return _flat(t, name, torch.int32, (n,), device)


def attention_cache_append(k, v, k_cache, v_cache, page_table, seqlens_k, cos=None, sin=None, positions=None, q=None, wq=None,
                           wk=None, eps: float = 1e-6, interleaved: bool = False, sections=None, cu_seqlens=None, q_out=None,
                           stream=None):
    """Appends k, v [T, Hk, d] to the paged cache, the keys normed (``wk``) and rotated (``cos``, ``sin``) on the way, and
    returns q normed and rotated the same way when it is given (else None).  ``seqlens_k`` holds the key counts after the
    append; ``cu_seqlens`` the sequences' rows (None: T/B each); ``positions`` those of the rotation (None: the positions in
    the cache)."""
    sk, sv = _rows(k, "k"), _rows(v, "v", k, k.shape[1])
    T, Hk, d = k.shape
    dev = k.device
    cd, chk, ps, pages, B, most, fmt = _cache(k_cache, v_cache, page_table)
    if (cd, chk) != (d, Hk) or k_cache.device != dev or (fmt == FA_CACHE_16BIT and k_cache.dtype != k.dtype):
        raise ValueError("the cache's heads, d, dtype and device must be those of k and v")
    lp = _lens(seqlens_k, "seqlens_k", B, dev)
    cu = None if cu_seqlens is None else _lens(cu_seqlens, "cu_seqlens", B + 1, dev)
    if q is None and wq is not None:
        raise ValueError("wq without q")
    if q is not None and (wq is None) != (wk is None):
        raise ValueError("norm weights come in pairs")
    w = _weights(wq, wk, d, k.dtype, dev)
    if cos is None and sin is None:
        if positions is not None or sections is not None:
            raise ValueError("positions and sections need cos and sin")
        rope = (None, None, None, 0, 0, 1, None)
    elif cos is None or sin is None:
        raise ValueError("cos and sin come in pairs")
    else:
        rope = _rope(cos, sin, positions, sections, T, dev)
    code = _code(k, "k")
    qp = op = None
    Hq = sq = so = 0
    if q is not None:
        sq, Hq = _rows(q, "q", k), q.shape[1]
        if q_out is None:
            q_out = _empty((T, Hq, d), q.dtype, dev, stream)
        so = _rows(q_out, "q_out", q, Hq)
        qp, op = q.data_ptr(), q_out.data_ptr()
    cp, sp, pp, rot, rows, axes, arr = rope
    _launch("fa_cache_append", lib.fa_cache_append, dev, stream, qp, k.data_ptr(), v.data_ptr(), op, k_cache.data_ptr(),
            v_cache.data_ptr(), w[0], w[1], cp, sp, pp, page_table.data_ptr(), lp, cu, B, T, Hq, Hk, d, sq, sk, sv, so, ps, pages,
            most, rot, rows, axes, arr, int(interleaved), float(eps), code, fmt)
    return q_out if q is not None else None


def attention_cache_gather(k_cache, v_cache, page_table, cu_seqlens_k, total_keys: int, starts=None, dtype=None, k=None, v=None,
                           stream=None):
    """(k, v) [total_keys, Hk, d]: rows cu_seqlens_k[b] .. cu_seqlens_k[b+1] hold positions starts[b], starts[b] + 1, … of
    sequence b (starts None: 0; cu_seqlens_k None: total_keys/B rows each).  ``dtype`` is needed for a 4-bit cache only."""
    d, Hk, ps, pages, B, most, fmt = _cache(k_cache, v_cache, page_table)
    dev = k_cache.device
    if fmt == FA_CACHE_16BIT:
        if dtype is not None and dtype != k_cache.dtype:
            raise ValueError("a 16-bit cache is read in its own dtype")
        dtype = k_cache.dtype
    elif dtype is None:
        dtype = k.dtype if k is not None else torch.bfloat16
    if dtype not in _CODES:
        raise TypeError(f"unsupported dtype {dtype}: k and v are bfloat16 or float16")
    total = int(total_keys)
    cu = None if cu_seqlens_k is None else _lens(cu_seqlens_k, "cu_seqlens_k", B + 1, dev)
    sp = None if starts is None else _lens(starts, "starts", B, dev)
    k = _empty((max(total, 0), Hk, d), dtype, dev, stream) if k is None else k
    v = _empty((max(total, 0), Hk, d), dtype, dev, stream) if v is None else v
    kp, vp = (_flat(t, n, dtype, (total, Hk, d), dev) for t, n in ((k, "k"), (v, "v")))
    _launch("fa_cache_gather", lib.fa_cache_gather, dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), kp, vp,
            page_table.data_ptr(), cu, sp, B, total, Hk, d, ps, pages, most, _CODES[dtype], fmt)
    return k, v


def attention_decode_paged(q, k_cache, v_cache, page_table, seqlens_k, max_seqlen_k: Optional[int] = None,
                           scale: Optional[float] = None, out=None, lse=None, workspace=None, stream=None):
    """O and LSE of the last tokens of each sequence over a paged cache: q [B, H, d] (one token each) or [B, Nq, H, d]; H a
    multiple of the cache's heads.  ``seqlens_k`` counts the keys, the new tokens' included; ``max_seqlen_k`` bounds them
    (None: the page table's capacity).  Query i of a sequence sees the keys up to position seqlens_k − Nq + i."""
    if q.dim() not in (3, 4) or not q.is_cuda or not q.is_contiguous():
        raise ValueError("q must be a contiguous CUDA tensor [B, H, d] or [B, Nq, H, d]")
    dev = q.device
    d, Hk, ps, pages, B, most, fmt = _cache(k_cache, v_cache, page_table)
    Nq = q.shape[1] if q.dim() == 4 else 1
    H = q.shape[-2]
    if q.shape[0] != B or q.shape[-1] != d or k_cache.device != dev or (fmt == FA_CACHE_16BIT and k_cache.dtype != q.dtype):
        raise ValueError("q's batch, d, dtype and device must be those of the page table and the cache")
    code = _code(q, "q")
    lp = _lens(seqlens_k, "seqlens_k", B, dev)
    Nk = most * ps if max_seqlen_k is None else int(max_seqlen_k)
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
        op = out.data_ptr()
    else:
        op = _flat(out, "out", q.dtype, q.shape, dev)
    if lse is None:
        lse = _empty(q.shape[:-1], torch.float32, dev, stream)
        ep = lse.data_ptr()
    else:
        ep = _flat(lse, "lse", torch.float32, q.shape[:-1], dev)
    if workspace is None:
        workspace = _empty((max(lib.fa_decode_paged_workspace_bytes(B, Nq, H, Hk, Nk, d), 256),), torch.uint8, dev, stream)
    _launch("fa_decode_paged", lib.fa_decode_paged, dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), op, ep,
            page_table.data_ptr(), lp, B, Nq, H, Hk, Nk, d, 1.0 / math.sqrt(d) if scale is None else float(scale), ps, pages, most,
            code, fmt, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse
