"""Binding of beam search over a hybrid decoder (``include/gdn_beam.h``): the selection of the
best continuations, and the reordering of recurrent states, page tables and pages after it.

Beam w of group (request) b is row b W + w wherever the beams of a call lie in one dimension.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _DT, _i, _vp, load
from .attention import _call, _device, _f32, _i32, _int32, _native

_i64 = ctypes.c_int64


class _Pool(ctypes.Structure):
    _fields_ = [("data", _vp), ("bytes", _i64), ("count", _i)]


class _Tables(ctypes.Structure):
    _fields_ = [("page_table", _vp), ("table_out", _vp), ("own_pages", _vp), ("kv_len", _vp),
                ("max_pages", _i), ("page_size", _i), ("table_stride", _i64), ("out_stride", _i64),
                ("own_stride", _i64)]


def _grid(name, t, B, W, dtypes, at):
    """[B, W] of one of `dtypes`, contiguous."""
    if t.shape != (B, W) or t.dtype not in dtypes or t.get_device() != at or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor [%d, %d] of %s on the call's device"
                         % (name, B, W, " or ".join(map(str, dtypes))))


def gdn_beam_select(logits, scores, n=None, *, done=None, eos=None, out=None, check=False):
    """The n (default: W) best continuations of every group of beams, best first: (scores fp32,
    beam int32, token int32), each [B, n].

    logits: [B, W, V] or [B * W, V], bf16 or fp32, rows the same distance apart; scores fp32
    [B, W], the beams' own, to which a token's log-probability is added.  done: bool or uint8
    [B, W], beams that go on with token `eos` alone, at the score that they have.  Equal scores go
    to the lowest (beam, token).  out: (scores, beam, token) to write."""
    if not check:
        r = _native().select(load().address["gdn_beam_select"], "gdn_beam_select", logits, scores, n,
                             done, eos, out)
        if r is not NotImplemented:
            return r
    at = _device("logits", logits)
    if scores.dim() != 2 or logits.dtype not in _DT or logits.dim() not in (2, 3):
        raise ValueError("logits must be [B, W, V] or [B * W, V], bf16 or fp32, and scores [B, W]")
    B, W = scores.shape
    V = logits.shape[-1]
    _grid("scores", scores, B, W, (_f32,), at)
    if logits.shape != ((B, W, V) if logits.dim() == 3 else (B * W, V)):
        raise ValueError("logits must have a row per score")
    if V > 1 and logits.stride(-1) != 1:
        raise ValueError("logits must have contiguous rows")
    stride = logits.stride(-2) if W > 1 or logits.dim() == 2 else logits.stride(0)
    if logits.dim() == 3 and B > 1 and W > 1 and logits.stride(0) != W * stride:
        raise ValueError("the rows of logits must be the same distance apart")
    if n is None:
        n = W
    if n < 1 or n > W * V:
        raise ValueError("there are %d continuations of a group to select from" % (W * V))
    if (done is None) != (eos is None):
        raise ValueError("done and eos go together")
    if done is not None:
        _grid("done", done, B, W, (torch.bool, torch.uint8), at)
        if not 0 <= eos < V:
            raise ValueError("eos must be a token")
    if out is None:
        out = (torch.empty((B, n), dtype=_f32, device=logits.device),
               torch.empty((B, n), dtype=_i32, device=logits.device),
               torch.empty((B, n), dtype=_i32, device=logits.device))
    else:
        for name, t, dtype in zip(("out[0]", "out[1]", "out[2]"), out, (_f32, _i32, _i32)):
            _grid(name, t, B, n, (dtype,), at)
    _call(load().gdn_beam_select, "gdn_beam_select", at, check, logits.data_ptr(), stride,
          scores.data_ptr(), None if done is None else done.data_ptr(), 0 if eos is None else eos,
          out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), B, W, V, n, _DT[logits.dtype])
    return out


# The structures packed into bytes, which costs a call less than filling ctypes ones.
_POOL, _TABLES = struct.Struct("@Pqi4x"), struct.Struct("@PPPPiiqqq")
assert (_POOL.size, _TABLES.size) == (ctypes.sizeof(_Pool), ctypes.sizeof(_Tables))


def _pools(name, tensors, at):
    pools = []
    for t in tensors:
        if t.dim() < 1 or t.get_device() != at or not t.is_contiguous():
            raise ValueError("%s must be contiguous tensors on the call's device" % name)
        n = t.shape[0]
        pools.append(_POOL.pack(t.data_ptr(), t.numel() // n * t.element_size() if n else 0, n))
    return b"".join(pools)


def gdn_beam_reorder(parent, slots, *, states=(), caches=(), page_table=None, own_pages=None,
                     kv_len=None, page_size=None, out=None, check=False):
    """Makes beam w of every group go on from beam parent[b, w] of it: returns the new slots
    [B, W], or (slots, page_table) where there is a page table.

    parent, slots: int32 [B, W]; slots are the lanes of the beams (distinct), rows of every tensor
    of `states` ([lanes, ...], what gdn_decode takes as state with these slots).  Of beams with the
    same parent the lowest keeps its lane, and nothing of it moves; the others take the lanes of
    beams that nobody goes on from, and their parent's states are copied there, in place.

    page_table int32 [B * W, pages], own_pages int32 [lanes, pages] (the pages that a lane may
    write), kv_len int32 [B * W] (a group's beams have the same) and page_size go together: full
    pages are shared by the tables, and of a page that is partly filled the others get a copy in
    every cache of `caches` (gdn_kv_pages, gdn_kv8_pages).  A sequence starts with table rows
    own_pages[slots].  out: slots, or (slots, page_table), to write; not the inputs."""
    if not check:
        r = _native().reorder(load().address["gdn_beam_reorder"], "gdn_beam_reorder", parent, slots,
                              states, caches, page_table, own_pages, kv_len, page_size, out)
        if r is not NotImplemented:
            return r
    at = _device("parent", parent)
    if parent.dim() != 2:
        raise ValueError("parent must be [B, W]")
    B, W = parent.shape
    _grid("parent", parent, B, W, (_i32,), at)
    _grid("slots", slots, B, W, (_i32,), at)
    states, caches = list(states), list(caches)
    tables = (page_table, own_pages, kv_len, page_size)
    paged = page_table is not None
    if any((t is not None) != paged for t in tables) or (caches and not paged):
        raise ValueError("page_table, own_pages, kv_len and page_size go together, and caches with them")
    if not states and not paged:
        raise ValueError("there is nothing to reorder: no states and no page table")
    rows = {t.shape[0] if t.dim() else -1 for t in states + ([own_pages] if paged else [])}
    lanes = rows.pop()
    if rows or lanes < 0:
        raise ValueError("states and own_pages must have a row per lane")
    new_slots, new_table = out if paged and out is not None else (out, None)
    if new_slots is None:
        new_slots = torch.empty((B, W), dtype=_i32, device=parent.device)
    else:
        _grid("out", new_slots, B, W, (_i32,), at)
    t = None
    if paged:
        _int32("page_table", page_table, 2, at)
        _int32("own_pages", own_pages, 2, at)
        _int32("kv_len", kv_len, 1, at)
        pages = page_table.shape[1]
        if new_table is None:
            new_table = torch.empty((B * W, pages), dtype=_i32, device=parent.device)
        else:
            _int32("out", new_table, 2, at)
        if page_table.shape[0] != B * W or new_table.shape != page_table.shape or \
                kv_len.shape[0] != B * W or own_pages.shape[1] != pages:
            raise ValueError("page_table and kv_len must have a row per beam, and page_table, "
                             "own_pages and out the same number of pages")
        t = _TABLES.pack(page_table.data_ptr(), new_table.data_ptr(), own_pages.data_ptr(),
                         kv_len.data_ptr(), pages, page_size, page_table.stride(0),
                         new_table.stride(0), own_pages.stride(0))
    if out is not None and B * W > 0:
        given = {x.data_ptr() for x in (parent, slots, page_table, own_pages, kv_len) if x is not None}
        if new_slots.data_ptr() in given or (paged and new_table.data_ptr() in given):
            raise ValueError("out cannot be an input")
    if lanes < 1 and B * W > 0:
        raise ValueError("there are no lanes")
    _call(load().gdn_beam_reorder, "gdn_beam_reorder", at, check, parent.data_ptr(),
          slots.data_ptr(), new_slots.data_ptr(), B, W, max(lanes, 1),
          _pools("states", states, at), len(states), t, _pools("caches", caches, at), len(caches))
    return (new_slots, new_table) if paged else new_slots
