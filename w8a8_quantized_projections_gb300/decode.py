"""Bindings for answering token by token: linears over 4-bit weights, the paged
8-bit cache of keys and values, its pages and the attention that reads it.

Like the rest of the binding this is argument marshalling: every function
checks placement, type, shape and layout (the C ABI receives bare pointers and
cannot see lengths), allocates outputs with torch where the caller passes none
and calls ``include/clef.h``.  Nothing here synchronises or reads the device.

A pool of pages is a pair of tensors: ``codes`` [planes][pages][heads][page][dim]
(``torch.int8``, or e4m3 as ``torch.uint8`` / ``torch.float8_e4m3fn``) and
``scales`` fp32 [planes][pages][heads].  A layer's two planes are its keys and its
values; calls that take a layer (append, gather, attention) take tensors of two
planes, such as ``codes[2 * layer : 2 * layer + 2]``; calls on pages take the whole pool.
``table`` int32 [sequences][width] and ``lens`` int32 [sequences] are shared by the
layers, ``refs`` int32 [pages] counts the sequences that hold each page.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math

import torch

from . import _FP8, _call, _cuda, _dense, _out_shape, _ptr, _rows, _stream

__all__ = ["quant_w4", "w4_linear", "kv_append", "kv_gather", "kv_attention", "kv_reserve", "kv_fork", "kv_free",
           "kv_compact", "kv_copy_pages"]

_INT8 = (torch.int8,)
_CODES = _INT8 + _FP8
_I32 = (torch.int32,)
_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)


def _scratch(shape, dtype, like, stream):
    """Scratch of a call on `stream`: torch's allocator hands memory out again
    in the order of the stream that was current at its allocation."""
    with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
        return torch.empty(shape, dtype=dtype, device=like.device)


def _same_device(first, *others):
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError("tensors on different devices")


# ---------------------------------------------------------------- 4-bit linears

def _w4_pad(K: int) -> int:
    return (K + 127) // 128 * 128


def quant_w4(w: torch.Tensor, group: int = 128, qw=None, sw=None, stream=None):
    """Packs bf16 weights [N][K] as 4-bit codes with a scale for each `group`
    (32, 64 or 128) weights of a row: (qw uint8 [N][K_pad / 2], sw bf16
    [N][K_pad / group]), K_pad = K rounded up to 128."""
    _cuda(w, "w", _BF16)
    ldw = _rows(w, "w")
    N, K = w.shape
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    Kp = _w4_pad(K)
    if qw is None:
        qw = _scratch((N, Kp // 2), torch.uint8, w, stream)
    if sw is None:
        sw = _scratch((N, Kp // group), torch.bfloat16, w, stream)
    _cuda(qw, "qw", (torch.uint8,)); _cuda(sw, "sw", _BF16)
    _dense(qw, "qw"); _dense(sw, "sw")
    if tuple(qw.shape) != (N, Kp // 2) or tuple(sw.shape) != (N, Kp // group):
        raise ValueError(f"qw must be {(N, Kp // 2)} and sw {(N, Kp // group)}")
    _same_device(w, qw, sw)
    _call("clef_quant_w4", _ptr(w), N, K, ldw, group, _ptr(qw), _ptr(sw), _stream(w, stream))
    return qw, sw


def w4_linear(x, qw, sw, bias=None, y=None, stream=None):
    """y = bf16(x W^T + bias) for bf16 x [M][K] and weights packed by quant_w4,
    for calls of few rows (weights are read once for every 16)."""
    _cuda(x, "x", _BF16); _cuda(qw, "qw", (torch.uint8,)); _cuda(sw, "sw", _BF16)
    ldx = _rows(x, "x")
    _dense(qw, "qw"); _dense(sw, "sw")
    if qw.dim() != 2 or sw.dim() != 2:
        raise ValueError("qw and sw must be 2-D")
    M, K = x.shape
    N, Kp = qw.shape[0], _w4_pad(K)
    if qw.shape[1] * 2 != Kp:
        raise ValueError(f"qw has {qw.shape[1]} bytes a row, x's {K} columns need {Kp // 2}")
    if sw.shape[0] != N or sw.shape[1] == 0 or Kp // sw.shape[1] not in (32, 64, 128) or Kp % sw.shape[1]:
        raise ValueError(f"sw has shape {tuple(sw.shape)}: one scale for each 32, 64 or 128 of {Kp} weights, {N} rows")
    if bias is not None:
        _cuda(bias, "bias", _BF16)
        _dense(bias, "bias")
        if bias.numel() != N:
            raise ValueError(f"bias has {bias.numel()} values for {N} weight rows")
    if y is None:
        y = _scratch((M, N), torch.bfloat16, x, stream)
    _cuda(y, "y", _BF16)
    _out_shape(y, M, N)
    _same_device(x, qw, sw, bias, y)
    _call("clef_w4_linear", _ptr(x), ldx, _ptr(qw), _ptr(sw), Kp // sw.shape[1], _ptr(bias), M, N, K, _ptr(y),
          _rows(y, "y"), _stream(x, stream))
    return y


# ---------------------------------------------------------------- arguments

def _pool(codes, scales, planes=None):
    """The C ABI's view of a pool: (codes, plane pitch, scales, plane pitch,
    planes, pages, heads, page, dim)."""
    _cuda(codes, "codes", _CODES); _cuda(scales, "scales", _F32)
    if codes.dim() > 5:
        codes, scales = codes.flatten(0, -5), scales.flatten(0, -3)
    if codes.dim() != 5 or tuple(scales.shape) != tuple(codes.shape[:3]):
        raise ValueError("codes must be [planes][pages][heads][page][dim] and scales [planes][pages][heads]")
    n, pages, heads, page, dim = codes.shape
    if planes is not None and n != planes:
        raise ValueError(f"codes has {n} planes, expected {planes} (a layer's keys, then its values)")
    if codes.numel() and (codes.stride()[1:] != (heads * page * dim, page * dim, dim, 1)
                          or scales.stride()[1:] != (heads, 1)):
        raise ValueError("each plane of codes and scales must be contiguous")
    _same_device(codes, scales)
    pc = codes.stride(0) if n > 1 else pages * heads * page * dim
    ps = scales.stride(0) if n > 1 else pages * heads
    return _ptr(codes), pc, _ptr(scales), ps, n, pages, heads, page, dim


def _kind(codes) -> int:
    return 0 if codes.dtype == torch.int8 else 1


def _table(table, lens=None):
    _cuda(table, "table", _I32)
    ldt = _rows(table, "table")
    if lens is not None:
        _ints(lens, "lens", table.shape[0])
        _same_device(table, lens)
    return ldt, table.shape[0], table.shape[1]


def _ints(t, name, n=None):
    _cuda(t, name, _I32)
    _dense(t, name)
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be int32 [{'n' if n is None else n}]")
    return t


def _heads(t, name, heads, dim):
    """Token and head pitch of a [tokens][heads][dim] tensor."""
    _cuda(t, name, _BF16)
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens][{heads if heads is not None else 'heads'}][{dim}], not {tuple(t.shape)}")
    if t.stride(2) != 1 and t.numel():
        raise ValueError(f"{name} must have contiguous heads")
    head = t.stride(1) if t.shape[1] > 1 else dim
    return (t.stride(0) if t.shape[0] > 1 else t.shape[1] * dim), head


def _row_start(row_start, rows, seqs):
    if row_start is None:
        if rows and (seqs == 0 or rows % seqs):
            raise ValueError(f"{rows} rows for {seqs} sequences: pass row_start, or the same number for each")
        return None
    return _ints(row_start, "row_start", seqs + 1)


# ---------------------------------------------------------------- cache

def kv_append(k, v, codes, scales, table, lens, row_start=None, stream=None) -> None:
    """Writes the newest tokens' keys and values (bf16 [tokens][heads][dim]) of
    one layer into the cache.  `lens` counts them already; a sequence's rows
    are its last tokens: rows row_start[b] .. row_start[b + 1] - 1, or the same
    number each."""
    pc = _pool(codes, scales, 2)
    heads, dim = pc[6], pc[8]
    ldk, ldk_head = _heads(k, "k", heads, dim)
    ldv, ldv_head = _heads(v, "v", heads, dim)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v differ in tokens")
    ldt, seqs, width = _table(table, lens)
    row_start = _row_start(row_start, k.shape[0], seqs)
    _same_device(codes, k, v, table, row_start)
    _call("clef_kv_append", _ptr(k), ldk, ldk_head, _ptr(v), ldv, ldv_head, k.shape[0], _ptr(row_start), _kind(codes),
          pc[0], pc[1], pc[2], pc[3], *pc[5:], _ptr(table), ldt, seqs, width, _ptr(lens), _stream(codes, stream))


def kv_gather(codes, scales, table, seq, pos, k=None, v=None, stream=None):
    """The keys and values that the cache of one layer stands for at token
    pos[r] of sequence seq[r]: bf16 (k, v), each [rows][heads][dim]."""
    pc = _pool(codes, scales, 2)
    heads, dim = pc[6], pc[8]
    _ints(seq, "seq")
    rows = seq.shape[0]
    _ints(pos, "pos", rows)
    ldt, seqs, width = _table(table)
    k = _scratch((rows, heads, dim), torch.bfloat16, codes, stream) if k is None else k
    v = _scratch((rows, heads, dim), torch.bfloat16, codes, stream) if v is None else v
    ld = []
    for t, name in ((k, "k"), (v, "v")):
        tok, head = _heads(t, name, heads, dim)
        if t.shape[0] != rows or head != dim:
            raise ValueError(f"{name} must have {rows} rows of contiguous heads")
        ld.append(tok)
    _same_device(codes, table, seq, pos, k, v)
    _call("clef_kv_gather", _kind(codes), pc[0], pc[1], pc[2], pc[3], *pc[5:], _ptr(table), ldt, seqs, width, _ptr(seq),
          _ptr(pos), rows, _ptr(k), ld[0], _ptr(v), ld[1], _stream(codes, stream))
    return k, v


def kv_attention(q, codes, scales, table, lens, row_start=None, scale=None, causal=True, out=None, lse=None,
                 stream=None):
    """Attention of bf16 queries [tokens][q_heads][dim] over the cache of one
    layer: the queries of a sequence are its last tokens (rows row_start[b] ..
    row_start[b + 1] - 1, or the same number each), query head h reads
    key/value head h // (q_heads // heads).  scale defaults to dim ** -0.5.
    Returns out, bf16 of q's shape; `lse` (fp32 [tokens][q_heads], optional)
    receives the log of each row's sum of exponentials.  A row that sees no
    token gives zeros (and minus infinity)."""
    pc = _pool(codes, scales, 2)
    heads, page, dim = pc[6:]
    ldq, ldq_head = _heads(q, "q", None, dim)
    rows, q_heads = q.shape[0], q.shape[1]
    if q_heads % heads or q_heads == 0:
        raise ValueError(f"{q_heads} query heads over {heads} key/value heads")
    ldt, seqs, width = _table(table, lens)
    row_start = _row_start(row_start, rows, seqs)
    if out is None:
        out = _scratch((rows, q_heads, dim), torch.bfloat16, q, stream)
    ldo, ldo_head = _heads(out, "out", q_heads, dim)
    if out.shape[0] != rows:
        raise ValueError(f"out has {out.shape[0]} rows, expected {rows}")
    # tokens of heads, or heads of tokens: either way the inner run has to fit between two of the outer
    if rows and not (ldo >= (q_heads - 1) * ldo_head + dim or ldo_head >= (rows - 1) * ldo + dim and ldo >= dim):
        raise ValueError("out's rows overlap")
    if lse is not None:
        _cuda(lse, "lse", _F32)
        _dense(lse, "lse")
        if tuple(lse.shape) != (rows, q_heads):
            raise ValueError(f"lse must be {(rows, q_heads)}")
    _same_device(q, codes, table, row_start, out, lse)
    need = C.c_int64(0)
    _call("clef_kv_attention_workspace", rows, int(row_start is not None), seqs, q_heads, heads, dim,
          min(width * page, 0x7FFFFFFF), C.byref(need))
    ws = _scratch((need.value,), torch.uint8, q, stream) if need.value else None
    _call("clef_kv_attention", _ptr(q), ldq, ldq_head, rows, _ptr(row_start), q_heads, _kind(codes), pc[0], pc[1], pc[2],
          pc[3], *pc[5:], _ptr(table), ldt, seqs, width, _ptr(lens), dim ** -0.5 if scale is None else float(scale),
          int(bool(causal)), _ptr(out), ldo, ldo_head, _ptr(lse), _ptr(ws), need.value, _stream(q, stream))
    return out


# ---------------------------------------------------------------- pages

def kv_reserve(table, lens, refs, grow, page: int, stream=None) -> None:
    """lens += grow (int32 [sequences]), with the pages of `page` tokens that
    takes: the lowest free ones, in the order of the sequences.  Changes
    nothing if the pool has too few (CLEF_ERR_NO_PAGES from poll_status)."""
    ldt, seqs, width = _table(table, lens)
    _ints(grow, "grow", seqs)
    _ints(refs, "refs")
    _same_device(table, refs, grow)
    _call("clef_kv_reserve", _ptr(table), ldt, seqs, width, _ptr(lens), _ptr(refs), refs.shape[0], int(page), _ptr(grow),
          _stream(table, stream))


def kv_fork(codes, scales, table, lens, refs, src, dst, stream=None) -> None:
    """Sequence dst[i] (empty before) becomes a copy of src[i]: whole pages are
    shared, a part-filled last page is copied to the lowest free page.  Changes
    nothing if the pool has too few free pages."""
    pc = _pool(codes, scales)
    ldt, seqs, width = _table(table, lens)
    _ints(refs, "refs", pc[5])
    _ints(src, "src")
    n = src.shape[0]
    _ints(dst, "dst", n)
    _same_device(codes, table, refs, src, dst)
    scratch = _scratch((2 * n,), torch.int32, table, stream)
    _call("clef_kv_fork", *pc, _ptr(table), ldt, seqs, width, _ptr(lens), _ptr(refs), _ptr(src), _ptr(dst), n,
          _ptr(scratch), _stream(table, stream))


def kv_free(table, lens, refs, seqs, page: int, stream=None) -> None:
    """The sequences listed in `seqs` (int32) give back their pages of `page`
    tokens and become empty."""
    ldt, count, width = _table(table, lens)
    _ints(refs, "refs")
    _ints(seqs, "seqs")
    _same_device(table, refs, seqs)
    _call("clef_kv_free", _ptr(table), ldt, count, width, _ptr(lens), _ptr(refs), refs.shape[0], int(page), _ptr(seqs),
          seqs.shape[0], _stream(table, stream))


def kv_compact(codes, scales, table, lens, refs, table_out=None, refs_out=None, stream=None):
    """Moves the held pages together at the pool's start and rewrites every
    sequence's row into table_out and refs into refs_out (in place where not
    given).  Returns the number of held pages, an int32 tensor of one value."""
    pc = _pool(codes, scales)
    ldt, seqs, width = _table(table, lens)
    table_out = table if table_out is None else table_out
    refs_out = refs if refs_out is None else refs_out
    _ints(refs, "refs", pc[5])
    _ints(refs_out, "refs_out", pc[5])
    ldt_out, s_out, w_out = _table(table_out)
    if (s_out, w_out) != (seqs, width):
        raise ValueError("table_out has another shape than table")
    _same_device(codes, table, refs, table_out, refs_out)
    live = _scratch((1,), torch.int32, table, stream)
    scratch = _scratch((3 * pc[5] + 1,), torch.int32, table, stream)
    if pc[5] == 0:
        live.zero_()
    _call("clef_kv_compact", *pc, _ptr(table), ldt, seqs, width, _ptr(lens), _ptr(refs), _ptr(table_out), ldt_out,
          _ptr(refs_out), _ptr(live), _ptr(scratch), _stream(table, stream))
    return live


def kv_copy_pages(codes, scales, src, dst, stream=None) -> None:
    """Page dst[i] becomes a copy of page src[i] (int32) in every plane; no
    target may also be a source or listed twice."""
    pc = _pool(codes, scales)
    _ints(src, "src")
    _ints(dst, "dst", src.shape[0])
    _same_device(codes, src, dst)
    _call("clef_kv_copy_pages", *pc, _ptr(src), _ptr(dst), src.shape[0], _stream(codes, stream))
