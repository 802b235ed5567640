"""Bindings for answering token by token: linears over 4-bit weights, the paged
8-bit cache of keys and values, its pages and the attention that reads it.

Like the rest of the binding this is argument marshalling, here in a compiled
module (``csrc/py_decode.cpp``): every function checks placement, type, shape
and layout, allocates outputs with torch where the caller passes none and calls
``include/clef.h``.  Nothing synchronises or reads the device.

A pool of pages is a pair of tensors: ``codes`` [planes][pages][heads][page][dim]
(``torch.int8``, or e4m3 as ``torch.uint8`` / ``torch.float8_e4m3fn``) and
``scales`` fp32 [planes][pages][heads].  A layer's two planes are its keys and its
values; calls that take a layer (append, gather, attention) take tensors of two
planes, such as ``codes[2 * layer : 2 * layer + 2]``; calls on pages take the whole pool.
``table`` int32 [sequences][width] and ``lens`` int32 [sequences] are shared by the
layers, ``refs`` int32 [pages] counts the sequences that hold each page.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util

import torch

from . import ClefError, _build, _lock, library

__all__ = ["quant_w4", "w4_linear", "kv_append", "kv_gather", "kv_attention", "kv_reserve", "kv_fork", "kv_free",
           "kv_compact", "kv_copy_pages"]

_ext = None


def _load():
    """The compiled module (built with the library on first use if absent or stale)."""
    global _ext
    library()
    with _lock:
        _build.build_extension()
    loader = importlib.machinery.ExtensionFileLoader("clef_decode", _build.EXT)
    ext = importlib.util.module_from_spec(importlib.util.spec_from_file_location("clef_decode", _build.EXT, loader=loader))
    loader.exec_module(ext)
    ext.set_error(ClefError)
    _ext = ext
    return ext


# ---------------------------------------------------------------- 4-bit linears

def quant_w4(w: torch.Tensor, group: int = 128, qw=None, sw=None, stream=None):
    """Packs bf16 weights [N][K] as 4-bit codes with a scale for each `group`
    (32, 64 or 128) weights of a row: (qw uint8 [N][K_pad / 2], sw bf16
    [N][K_pad / group]), K_pad = K rounded up to 128."""
    return (_ext or _load()).quant_w4(w, group, qw, sw, stream)


def w4_linear(x, qw, sw, bias=None, y=None, stream=None):
    """y = bf16(x W^T + bias) for bf16 x [M][K] and weights packed by quant_w4,
    for calls of few rows (weights are read once for every 16, or every 8 of
    the largest K)."""
    return (_ext or _load()).w4_linear(x, qw, sw, bias, y, stream)


# ---------------------------------------------------------------- cache

def kv_append(k, v, codes, scales, table, lens, row_start=None, stream=None) -> None:
    """Writes the newest tokens' keys and values (bf16 [tokens][heads][dim]) of
    one layer into the cache.  `lens` counts them already; a sequence's rows
    are its last tokens: rows row_start[b] .. row_start[b + 1] - 1, or the same
    number each.  Where the pool may be full, take row_start from kv_reserve.
    A page has one scale a head, so values written one by one are off by more
    than those of a page written at once (include/clef.h has the bound)."""
    (_ext or _load()).kv_append(k, v, codes, scales, table, lens, row_start, stream)


def kv_gather(codes, scales, table, seq, pos, k=None, v=None, stream=None):
    """The keys and values that the cache of one layer stands for at token
    pos[r] of sequence seq[r]: bf16 (k, v), each [rows][heads][dim].  The call is
    not told the lengths: a position past a sequence's tokens gives whatever its
    place last held."""
    return (_ext or _load()).kv_gather(codes, scales, table, seq, pos, k, v, stream)


def kv_attention(q, codes, scales, table, lens, row_start=None, scale=None, causal=True, out=None, lse=None,
                 stream=None):
    """Attention of bf16 queries [tokens][q_heads][dim] over the cache of one
    layer: the queries of a sequence are its last tokens (rows row_start[b] ..
    row_start[b + 1] - 1, or the same number each), query head h reads
    key/value head h // (q_heads // heads).  scale defaults to dim ** -0.5.
    Returns out, bf16 of q's shape; `lse` (fp32 [tokens][q_heads], optional)
    receives the log of each row's sum of exponentials.  A row that sees no
    token gives zeros (and minus infinity)."""
    return (_ext or _load()).kv_attention(q, codes, scales, table, lens, row_start, scale, causal, out, lse, stream)


# ---------------------------------------------------------------- pages

def kv_reserve(table, lens, refs, grow, page: int, stream=None, row_start=None) -> None:
    """lens += grow (int32 [sequences]), with the pages of `page` tokens that
    takes: the lowest free ones, in the order of the sequences.  Changes
    nothing if the pool has too few (CLEF_ERR_NO_PAGES from poll_status).
    `row_start` (int32 [sequences + 1], optional) receives the running sum of
    grow, or zeros if nothing was reserved: kv_append with it then writes
    nothing, where it would write over the last tokens otherwise."""
    (_ext or _load()).kv_reserve(table, lens, refs, grow, page, stream, row_start)


def kv_fork(codes, scales, table, lens, refs, src, dst, stream=None) -> None:
    """Sequence dst[i] (empty before) becomes a copy of src[i] as it was before the
    call: whole pages are shared, a part-filled last page is copied to the lowest free page.  Changes
    nothing if the pool has too few free pages."""
    (_ext or _load()).kv_fork(codes, scales, table, lens, refs, src, dst, stream)


def kv_free(table, lens, refs, seqs, page: int, stream=None) -> None:
    """The sequences listed in `seqs` (int32) give back their pages of `page`
    tokens and become empty."""
    (_ext or _load()).kv_free(table, lens, refs, seqs, page, stream)


def kv_compact(codes, scales, table, lens, refs, table_out=None, refs_out=None, stream=None):
    """Moves the held pages together at the pool's start and rewrites every
    sequence's row into table_out and refs into refs_out (in place where not
    given).  Returns the number of held pages, an int32 tensor of one value."""
    return (_ext or _load()).kv_compact(codes, scales, table, lens, refs, table_out, refs_out, stream)


def kv_copy_pages(codes, scales, src, dst, stream=None) -> None:
    """Page dst[i] becomes a copy of page src[i] (int32) in every plane; no
    target may also be a source or listed twice."""
    (_ext or _load()).kv_copy_pages(codes, scales, src, dst, stream)
