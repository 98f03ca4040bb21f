"""Binding of the softmax-attention layers of a hybrid decoder
(``include/gdn_attn.h``): rotary positions, a paged key/value cache held in 4
bits, and attention over that cache.

Rows are found by strides: q, k, v and o may be any views whose last dimension
is contiguous ([tokens, heads, d], or a transposed [heads, tokens, d]).  The
cache entry points take the last tokens of each sequence, packed; ``kv_len``
counts a sequence's tokens including them.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _DT, GdnError, _check, _i, _stream, _vp, load

GDN_ROPE_ADJACENT = 1
GDN_ROPE_INVERSE = 2
GDN_ATTN_CAUSAL = 1

_i64 = ctypes.c_int64


class _Rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("stride_seq", _i64), ("stride_head", _i64), ("stride_tok", _i64),
                ("heads", _i)]


class _Rotary(ctypes.Structure):
    _fields_ = [("cos", _vp), ("sin", _vp), ("pos", _vp), ("axes", ctypes.c_char_p),
                ("stride_axis", _i64), ("stride_seq", _i64), ("table_len", _i), ("d_rot", _i),
                ("n_axes", _i), ("flags", ctypes.c_uint)]


class _Kv(ctypes.Structure):
    _fields_ = [("pages", _vp), ("head_scale", _vp), ("page_table", _vp), ("kv_len", _vp),
                ("cu_seqlens", _vp), ("n_pages", _i), ("page_size", _i), ("heads", _i), ("d", _i),
                ("N", _i), ("max_pages", _i), ("n_tokens", _i), ("table_stride", _i64)]


# The same structures packed into bytes, which costs a call less than filling a ctypes one (a
# single token's call is bound by the host).
_ROWS = struct.Struct("@Pqqqi4x")
_ROTARY = struct.Struct("@PPPPqqiiiI")
_KV = struct.Struct("@PPPPPiiiiiii4xq")
assert (_ROWS.size, _ROTARY.size, _KV.size) == tuple(map(ctypes.sizeof, (_Rows, _Rotary, _Kv)))

_f32, _i32, _u8 = torch.float32, torch.int32, torch.uint8
_INT_MAX = 2 ** 31 - 1     # (larger bounds and windows mean the same)
_axes_kept: dict = {}      # axis numbers by their value, as C arrays


def _device(name, t):
    """The GPU of the call, that of t."""
    at = t.get_device()
    if at < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    return at


def _rows3(name, t, heads, n, d, dtype, at):
    """[tokens, heads, d] rows."""
    tok, head, one = t.stride()
    if t.shape != (n, heads, d) or one != 1 or t.dtype != dtype or t.get_device() != at:
        raise ValueError("%s must be a CUDA tensor [tokens, heads, d] of the call's dtype and "
                         "device, its last dimension contiguous" % name)
    # (a dimension of one entry may have any stride)
    return _ROWS.pack(t.data_ptr(), 0, head if heads > 1 else 0, tok if n > 1 else 0, heads)


def _rows4(name, t, like, heads, at):
    """[B, heads, T, d] rows, like's but for the heads."""
    B, _, T, d = like.shape
    if t.shape != (B, heads, T, d) or t.stride(3) != 1 or t.dtype != like.dtype or \
            t.get_device() != at:
        raise ValueError("%s must be a CUDA tensor [B, heads, T, d] of the call's dtype and "
                         "device, its last dimension contiguous" % name)
    seq, head, tok, _ = t.stride()
    return _ROWS.pack(t.data_ptr(), seq if B > 1 else 0, head if heads > 1 else 0,
                      tok if T > 1 else 0, heads)


def _int32(name, t, dims, at):
    if t.dim() != dims or t.dtype != _i32 or t.get_device() != at or \
            (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError("%s must be a %d-D int32 tensor on the call's device, its last dimension "
                         "contiguous" % (name, dims))


def _rotary(cos, sin, pos, axes, flags, shape, at):
    """shape: the shape that one axis of `pos` has, or may have without its first part."""
    table = cos.shape
    if cos.dim() != 2 or table != sin.shape or cos.dtype != _f32 or sin.dtype != _f32 or \
            cos.get_device() != at or sin.get_device() != at or not cos.is_contiguous() or \
            not sin.is_contiguous():
        raise ValueError("cos and sin must be contiguous fp32 tensors [positions, d_rot / 2] on "
                         "the call's device")
    lead = 0 if axes is None else 1
    whole = pos.dim() == lead + len(shape)
    _int32("pos", pos, lead + (len(shape) if whole else 1), at)
    if pos.shape[lead:] != (shape if whole else shape[-1:]):
        raise ValueError("pos must hold a position per token%s" % (" on each axis" if lead else ""))
    axes_at = 0
    if lead:
        axes = bytes(axes)
        if len(axes) != table[1]:
            raise ValueError("axes must give the axis of each of the d_rot / 2 pairs")
        kept = _axes_kept.get(axes)
        if kept is None:
            kept = _axes_kept[axes] = ctypes.create_string_buffer(axes, max(1, len(axes)))
        axes_at = ctypes.addressof(kept)
    return _ROTARY.pack(cos.data_ptr(), sin.data_ptr(), pos.data_ptr(), axes_at,
                        pos.stride(0) if lead else 0,
                        pos.stride(lead) if whole and len(shape) == 2 else 0, table[0],
                        2 * table[1], pos.shape[0] if lead else 1, flags)


def _kv(pages, page_table, kv_len, cu_seqlens, kv_scale, n_tokens, d, at):
    """The packed gdn_kv, and the cache's heads and page size."""
    if pages.dim() != 3 or pages.dtype != _u8 or pages.get_device() != at or \
            not pages.is_contiguous():
        raise ValueError("pages must be a contiguous uint8 tensor [n_pages, heads, page bytes] on "
                         "the call's device")
    n_pages, heads, size = pages.shape
    page_size = size * 8 // (9 * d) if d > 0 else 0
    if page_size * d * 9 != size * 8 or page_size < 1:
        raise ValueError("a page of %d bytes does not hold rows of d = %d" % (size, d))
    _int32("page_table", page_table, 2, at)
    _int32("kv_len", kv_len, 1, at)
    N, (rows, max_pages) = kv_len.shape[0], page_table.shape
    if rows != N:
        raise ValueError("page_table must have a row per sequence")
    cu = 0
    if cu_seqlens is not None:
        _int32("cu_seqlens", cu_seqlens, 1, at)
        if cu_seqlens.shape[0] != N + 1:
            raise ValueError("cu_seqlens must have one entry more than there are sequences")
        cu = cu_seqlens.data_ptr()
    elif n_tokens < 0 or n_tokens and (N == 0 or n_tokens % N):
        raise ValueError("without cu_seqlens every sequence has the same number of tokens")
    scale = 0
    if kv_scale is not None:
        if kv_scale.shape != (2, heads) or kv_scale.dtype != _f32 or \
                kv_scale.get_device() != at or not kv_scale.is_contiguous():
            raise ValueError("kv_scale must be a contiguous fp32 tensor [2, heads] on the call's "
                             "device")
        scale = kv_scale.data_ptr()
    return _KV.pack(pages.data_ptr(), scale, page_table.data_ptr(), kv_len.data_ptr(), cu, n_pages,
                    page_size, heads, d, N, max_pages, n_tokens, page_table.stride(0)), \
        heads, page_size


def _call(fn, what, at, check, *args):
    """fn(*args, stream) on GPU `at` and its current stream."""
    if torch._C._cuda_getDevice() != at:
        with torch.cuda.device(at):
            return _call(fn, what, at, check, *args)
    rc = fn(*args, torch._C._cuda_getCurrentRawStream(at))
    if rc:
        raise GdnError(rc, what)
    if check:
        _check(load().gdn_sync_check(_stream(at)), what + " (device)")


def gdn_kv_page_bytes(page_size: int, d: int) -> int:
    """Bytes of one page of one head; 0 where the sizes are not supported."""
    return int(load().gdn_kv_page_bytes(int(page_size), int(d)))


def gdn_kv_pages(n_pages, heads, page_size, d, device=None):
    """A new cache: uint8 [n_pages, heads, page bytes], zeroed."""
    size = gdn_kv_page_bytes(page_size, d)
    if size == 0:
        raise ValueError("page_size must be 16, 32, 64, 128 or 256 and d 64, 128 or 256")
    return torch.zeros((n_pages, heads, size), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def gdn_rope_table(n_pos, d_rot, base=10000.0, device=None):
    """(cos, sin), fp32 [n_pos, d_rot / 2], of position * base^(-2 i / d_rot), formed in fp64."""
    if n_pos < 0 or d_rot < 0 or d_rot % 2:
        raise ValueError("a table has n_pos >= 0 positions of d_rot / 2 pairs")
    device = "cuda" if device is None else device
    f = torch.exp(torch.arange(0, d_rot, 2, dtype=torch.float64, device=device)
                  * (-math.log(base) / max(d_rot, 1)))
    a = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * f
    return a.cos().float(), a.sin().float()


def gdn_rope_axes(sections, interleave=False):
    """The axis of each pair, for `axes`: sections[a] pairs go by axis a, in runs, or dealt out
    in turn as long as an axis has some left."""
    left = list(sections)
    if any(n < 0 for n in left):
        raise ValueError("sections are numbers of pairs")
    if not interleave:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return bytes(out)


def _rope(q, k, cos, sin, pos, axes, flags, out, check, what):
    if q.dtype not in _DT or q.dim() != 4:
        raise ValueError("q must be [B, heads, T, d], bf16 or fp32")
    at = _device("q", q)
    B, Hq, T, d = q.shape
    qo, ko = out if out is not None else (torch.empty_like(q),
                                          None if k is None else torch.empty_like(k))
    rk = rko = None
    if (k is None) != (ko is None):
        raise ValueError("out must hold a place for k where there is a k, and None elsewhere")
    if k is not None:
        Hk = k.shape[1] if k.dim() == 4 else 0
        rk, rko = _rows4("k", k, q, Hk, at), _rows4("out[1]", ko, q, Hk, at)
    _call(load().gdn_rope, what, at, check, _rows4("q", q, q, Hq, at),
          _rows4("out[0]", qo, q, Hq, at), rk, rko, B, T, d,
          _rotary(cos, sin, pos, axes, flags, (B, T), at), _DT[q.dtype])
    return qo, ko


def gdn_rope(q, k, cos, sin, pos, *, axes=None, adjacent=False, out=None, check=False):
    """Turns q [B, Hq, T, d] and k [B, Hk, T, d] (or None) by their positions: returns (q, k).

    cos, sin: fp32 [positions, d_rot / 2] (gdn_rope_table); pos int32 [T] or [B, T].  With
    several axes, `axes` gives the axis of each pair (gdn_rope_axes) and pos is [axes, T] or
    [axes, B, T].  adjacent: pairs (2 i, 2 i + 1) instead of (i, i + d_rot / 2).  out: (q, k) to
    write, which may be the inputs."""
    return _rope(q, k, cos, sin, pos, axes, GDN_ROPE_ADJACENT if adjacent else 0, out, check,
                 "gdn_rope")


def gdn_rope_bwd(dq, dk, cos, sin, pos, *, axes=None, adjacent=False, out=None, check=False):
    """The gradient of gdn_rope with respect to q and k, from that of its results."""
    return _rope(dq, dk, cos, sin, pos, axes,
                 GDN_ROPE_INVERSE | (GDN_ROPE_ADJACENT if adjacent else 0), out, check,
                 "gdn_rope_bwd")


def gdn_kv_append(pages, k, v, page_table, kv_len, *, q=None, cu_seqlens=None, kv_scale=None,
                  cos=None, sin=None, pos=None, axes=None, adjacent=False, out=None, check=False):
    """Appends k, v [tokens, heads, d] to the cache, k turned by its positions (where cos, sin
    and pos int32 [tokens], or [axes, tokens], are given), and returns q [tokens, Hq, d] turned
    likewise (None without q).

    pages: the cache (gdn_kv_pages), written in place; page_table int32 [N, pages]; kv_len int32
    [N], the sequences' tokens with the new ones; cu_seqlens int32 [N + 1] or None for the same
    number of new tokens each; kv_scale fp32 [2, heads]: a further scale per head."""
    if k.dtype not in _DT or k.dim() != 3:
        raise ValueError("k must be [tokens, heads, d], bf16 or fp32")
    at = _device("k", k)
    n, _, d = k.shape
    dtype = k.dtype
    kv, heads, _ = _kv(pages, page_table, kv_len, cu_seqlens, kv_scale, n, d, at)
    rq = rqo = rot = None
    if cos is None or sin is None or pos is None:
        if adjacent or any(x is not None for x in (cos, sin, pos, axes)):
            raise ValueError("cos, sin and pos go together, and axes and adjacent with them")
    if q is None and out is not None:
        raise ValueError("out is where q goes, and there is no q")
    if q is not None:
        if out is None:
            out = torch.empty_like(q)
        Hq = q.shape[1] if q.dim() == 3 else 0
        rq, rqo = _rows3("q", q, Hq, n, d, dtype, at), _rows3("out", out, Hq, n, d, dtype, at)
    if cos is not None:
        rot = _rotary(cos, sin, pos, axes, GDN_ROPE_ADJACENT if adjacent else 0, (n,), at)
    _call(load().gdn_kv_append, "gdn_kv_append", at, check, kv,
          _rows3("k", k, heads, n, d, dtype, at), _rows3("v", v, heads, n, d, dtype, at), rq, rqo,
          rot, _DT[dtype])
    return out if q is not None else None


def gdn_kv_read(pages, page_table, kv_len, n_tokens, d, *, cu_seqlens=None, kv_scale=None,
                dtype=torch.bfloat16, out=None, check=False):
    """The last n_tokens tokens (packed as in gdn_kv_append) back from the cache, as the values
    they are held as: (k, v), each [tokens, heads, d] of `dtype`."""
    if dtype not in _DT:
        raise ValueError("k and v are read as bf16 or fp32")
    at = _device("pages", pages)
    kv, heads, _ = _kv(pages, page_table, kv_len, cu_seqlens, kv_scale, n_tokens, d, at)
    if out is None:
        k = torch.empty((n_tokens, heads, d), dtype=dtype, device=pages.device)
        v = torch.empty_like(k)
    else:
        k, v = out
    _call(load().gdn_kv_read, "gdn_kv_read", at, check, kv,
          _rows3("out", k, heads, n_tokens, d, dtype, at),
          _rows3("out", v, heads, n_tokens, d, dtype, at), _DT[dtype])
    return k, v


def gdn_kv_attn(q, pages, page_table, kv_len, *, cu_seqlens=None, kv_scale=None, max_len=None,
                max_new=None, scale=None, causal=True, window=0, out=None, return_lse=False,
                check=False):
    """Attention of the last tokens of each sequence, q [tokens, Hq, d] (turned already), over
    the cached keys and values: o like q, or (o, lse fp32 [tokens, Hq]).

    The cache arguments as in gdn_kv_append, after the append.  max_len and max_new: bounds on
    kv_len and on a sequence's tokens in this call, known on the host (default: what the page
    table holds, and the same number of tokens each, or with cu_seqlens all of the call's); they
    plan the launch and choose its kernel.  A decode step that carries cu_seqlens should pass
    max_new=1: without it the call is planned for one sequence that has all the tokens.  scale:
    default d^-1/2.  window: a token sees the last `window` places up to its own (0: all)."""
    if q.dtype not in _DT or q.dim() != 3:
        raise ValueError("q must be [tokens, heads, d], bf16 or fp32")
    at = _device("q", q)
    n, Hq, d = q.shape
    dtype = q.dtype
    kv, _, page_size = _kv(pages, page_table, kv_len, cu_seqlens, kv_scale, n, d, at)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((n, Hq), dtype=_f32, device=q.device) if return_lse else None
    if max_len is None:
        max_len = page_table.shape[1] * page_size
    if max_new is None:
        max_new = n if cu_seqlens is not None else n // max(kv_len.shape[0], 1)
    _call(load().gdn_kv_attn, "gdn_kv_attn", at, check, kv, _rows3("q", q, Hq, n, d, dtype, at),
          _rows3("out", out, Hq, n, d, dtype, at), None if lse is None else lse.data_ptr(),
          min(max_len, _INT_MAX), min(max_new, _INT_MAX), d ** -0.5 if scale is None else scale,
          min(window, _INT_MAX), GDN_ATTN_CAUSAL if causal else 0, _DT[dtype])
    return (out, lse) if return_lse else out
