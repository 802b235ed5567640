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

import ctypes as C
import functools

import torch

from . import ClefError, library

__all__ = ["quant_w4", "w4_linear", "kv_append", "kv_gather", "kv_attention", "kv_reserve", "kv_fork", "kv_free",
           "kv_compact", "kv_copy_pages"]

_BF16, _F32, _I32, _U8, _I8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int8
_CODES = (torch.int8, torch.uint8, torch.float8_e4m3fn)

# A single-token call runs for a few microseconds on the device, so the binding keeps its own part short: one
# attribute read a check, no wrapper objects, the current stream by its handle.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


@functools.lru_cache(maxsize=None)
def _function(name):
    return getattr(library(), name)


def _call(name, *args):
    rc = _function(name)(*args)
    if rc != 0:
        raise ClefError(name, rc, library().clef_last_error().decode(errors="replace"))


def _handle(device: int, stream):
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _new(shape, dtype, device, stream):
    """An output or scratch tensor of a call on `stream`: torch's allocator hands
    memory out again in the order of the stream that was current at its allocation."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _on(t, name, dtype, device=None) -> int:
    """Checks type and place; the device's index."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    index = t.get_device()
    if device is not None and index != device:
        raise ValueError(f"{name} is on device {index}, other tensors on {device}")
    return index


def _pitch(t, name) -> int:
    """Row pitch of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ---------------------------------------------------------------- 4-bit linears

def _w4_pad(K: int) -> int:
    return (K + 127) // 128 * 128


def quant_w4(w: torch.Tensor, group: int = 128, qw=None, sw=None, stream=None):
    """Packs bf16 weights [N][K] as 4-bit codes with a scale for each `group`
    (32, 64 or 128) weights of a row: (qw uint8 [N][K_pad / 2], sw bf16
    [N][K_pad / group]), K_pad = K rounded up to 128."""
    dev = _on(w, "w", _BF16)
    ldw = _pitch(w, "w")
    N, K = w.shape
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    Kp = _w4_pad(K)
    if qw is None:
        qw = _new((N, Kp // 2), _U8, w.device, stream)
    if sw is None:
        sw = _new((N, Kp // group), _BF16, w.device, stream)
    _on(qw, "qw", _U8, dev)
    _on(sw, "sw", _BF16, dev)
    _dense(qw, "qw")
    _dense(sw, "sw")
    if qw.shape != (N, Kp // 2) or sw.shape != (N, Kp // group):
        raise ValueError(f"qw must be {(N, Kp // 2)} and sw {(N, Kp // group)}")
    _call("clef_quant_w4", w.data_ptr(), N, K, ldw, group, qw.data_ptr(), sw.data_ptr(), _handle(dev, stream))
    return qw, sw


def w4_linear(x, qw, sw, bias=None, y=None, stream=None):
    """y = bf16(x W^T + bias) for bf16 x [M][K] and weights packed by quant_w4,
    for calls of few rows (weights are read once for every 16)."""
    dev = _on(x, "x", _BF16)
    _on(qw, "qw", _U8, dev)
    _on(sw, "sw", _BF16, dev)
    ldx = _pitch(x, "x")
    _dense(qw, "qw")
    _dense(sw, "sw")
    if qw.dim() != 2 or sw.dim() != 2:
        raise ValueError("qw and sw must be 2-D")
    M, K = x.shape
    N, row_bytes = qw.shape
    Kp = (K + 127) // 128 * 128
    if row_bytes * 2 != Kp:
        raise ValueError(f"qw has {row_bytes} bytes a row, x's {K} columns need {Kp // 2}")
    rows, scales = sw.shape
    group = Kp // scales if scales else 0
    if rows != N or group not in (32, 64, 128) or group * scales != Kp:
        raise ValueError(f"sw has shape {tuple(sw.shape)}: one scale for each 32, 64 or 128 of {Kp} weights, {N} rows")
    if bias is not None:
        _on(bias, "bias", _BF16, dev)
        _dense(bias, "bias")
        if bias.numel() != N:
            raise ValueError(f"bias has {bias.numel()} values for {N} weight rows")
    if y is None:
        y, ldy = _new((M, N), _BF16, x.device, stream), N
    else:
        _on(y, "y", _BF16, dev)
        if y.shape != (M, N):
            raise ValueError(f"output has shape {tuple(y.shape)}, expected ({M}, {N})")
        ldy = _pitch(y, "y")
    _call("clef_w4_linear", x.data_ptr(), ldx, qw.data_ptr(), sw.data_ptr(), group, None if bias is None else bias.data_ptr(),
          M, N, K, y.data_ptr(), ldy, _handle(dev, stream))
    return y


# ---------------------------------------------------------------- arguments

def _pool(codes, scales, planes=None):
    """The C ABI's view of a pool: (codes, plane pitch, scales, plane pitch,
    planes, pages, heads, page, dim), and the device's index."""
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda:
        raise ValueError("codes must be a CUDA tensor")
    if codes.dtype not in _CODES:
        raise ValueError(f"codes has dtype {codes.dtype}, expected one of {_CODES}")
    dev = codes.get_device()
    _on(scales, "scales", _F32, dev)
    if codes.dim() > 5:
        codes, scales = codes.flatten(0, -5), scales.flatten(0, -3)
    if codes.dim() != 5 or scales.dim() != 3 or scales.shape != codes.shape[:3]:
        raise ValueError("codes must be [planes][pages][heads][page][dim] and scales [planes][pages][heads]")
    n, pages, heads, page, dim = codes.shape
    if planes is not None and n != planes:
        raise ValueError(f"codes has {n} planes, expected {planes} (a layer's keys, then its values)")
    pc, ps = codes.stride(), scales.stride()
    tile = page * dim
    if pages and heads and tile and (pc[1:] != (heads * tile, tile, dim, 1) or ps[1:] != (heads, 1)):
        raise ValueError("each plane of codes and scales must be contiguous")
    return (codes.data_ptr(), pc[0] if n > 1 else pages * heads * tile, scales.data_ptr(),
            ps[0] if n > 1 else pages * heads, n, pages, heads, page, dim), dev


def _table(table, lens, dev):
    _on(table, "table", _I32, dev)
    if lens is not None:
        _ints(lens, "lens", dev, table.shape[0])
    ldt = _pitch(table, "table")
    seqs, width = table.shape
    return ldt, seqs, width


def _ints(t, name, dev, n=None):
    _on(t, name, _I32, dev)
    if t.dim() != 1 or (n is not None and t.shape[0] != n) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 [{'n' if n is None else n}]")
    return t.data_ptr()


def _heads(t, name, dev, heads, dim):
    """Token and head pitch of a [tokens][heads][dim] tensor."""
    _on(t, name, _BF16, dev)
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens][{heads if heads is not None else 'heads'}][{dim}], not {tuple(t.shape)}")
    tokens, count, _ = t.shape
    tok, head, one = t.stride()
    if one != 1 and t.numel():
        raise ValueError(f"{name} must have contiguous heads")
    if count == 1:
        head = dim
    return (tok if tokens > 1 else count * dim), head


def _row_start(row_start, rows, seqs, dev):
    if row_start is None:
        if rows and (seqs == 0 or rows % seqs):
            raise ValueError(f"{rows} rows for {seqs} sequences: pass row_start, or the same number for each")
        return None
    return _ints(row_start, "row_start", dev, seqs + 1)


# ---------------------------------------------------------------- cache

def kv_append(k, v, codes, scales, table, lens, row_start=None, stream=None) -> None:
    """Writes the newest tokens' keys and values (bf16 [tokens][heads][dim]) of
    one layer into the cache.  `lens` counts them already; a sequence's rows
    are its last tokens: rows row_start[b] .. row_start[b + 1] - 1, or the same
    number each."""
    (c, pc, sc, ps, _, pages, heads, page, dim), dev = _pool(codes, scales, 2)
    ldk, ldk_head = _heads(k, "k", dev, heads, dim)
    ldv, ldv_head = _heads(v, "v", dev, heads, dim)
    rows = k.shape[0]
    if rows != v.shape[0]:
        raise ValueError("k and v differ in tokens")
    ldt, seqs, width = _table(table, lens, dev)
    _call("clef_kv_append", k.data_ptr(), ldk, ldk_head, v.data_ptr(), ldv, ldv_head, rows,
          _row_start(row_start, rows, seqs, dev), 0 if codes.dtype is _I8 else 1, c, pc, sc, ps, pages, heads, page, dim,
          table.data_ptr(), ldt, seqs, width, lens.data_ptr(), _handle(dev, stream))


def kv_gather(codes, scales, table, seq, pos, k=None, v=None, stream=None):
    """The keys and values that the cache of one layer stands for at token
    pos[r] of sequence seq[r]: bf16 (k, v), each [rows][heads][dim]."""
    (c, pc, sc, ps, _, pages, heads, page, dim), dev = _pool(codes, scales, 2)
    seq_at = _ints(seq, "seq", dev)
    rows = seq.shape[0]
    pos_at = _ints(pos, "pos", dev, rows)
    ldt, seqs, width = _table(table, None, dev)
    ld = []
    if k is None:
        k = _new((rows, heads, dim), _BF16, codes.device, stream)
    if v is None:
        v = _new((rows, heads, dim), _BF16, codes.device, stream)
    for t, name in ((k, "k"), (v, "v")):
        tok, head = _heads(t, name, dev, heads, dim)
        if t.shape[0] != rows or head != dim:
            raise ValueError(f"{name} must have {rows} rows of contiguous heads")
        ld.append(tok)
    _call("clef_kv_gather", 0 if codes.dtype is _I8 else 1, c, pc, sc, ps, pages, heads, page, dim, table.data_ptr(), ldt,
          seqs, width, seq_at, pos_at, rows, k.data_ptr(), ld[0], v.data_ptr(), ld[1], _handle(dev, stream))
    return k, v


@functools.lru_cache(maxsize=4096)
def _attention_workspace(*shape) -> int:
    """Bytes that a call of these sizes needs (a function of the sizes alone)."""
    need = C.c_int64(0)
    _call("clef_kv_attention_workspace", *shape, C.byref(need))
    return need.value


def kv_attention(q, codes, scales, table, lens, row_start=None, scale=None, causal=True, out=None, lse=None,
                 stream=None):
    """Attention of bf16 queries [tokens][q_heads][dim] over the cache of one
    layer: the queries of a sequence are its last tokens (rows row_start[b] ..
    row_start[b + 1] - 1, or the same number each), query head h reads
    key/value head h // (q_heads // heads).  scale defaults to dim ** -0.5.
    Returns out, bf16 of q's shape; `lse` (fp32 [tokens][q_heads], optional)
    receives the log of each row's sum of exponentials.  A row that sees no
    token gives zeros (and minus infinity)."""
    (c, pc, sc, ps, _, pages, heads, page, dim), dev = _pool(codes, scales, 2)
    ldq, ldq_head = _heads(q, "q", dev, None, dim)
    rows, q_heads, _ = q.shape
    if q_heads % heads or q_heads == 0:
        raise ValueError(f"{q_heads} query heads over {heads} key/value heads")
    ldt, seqs, width = _table(table, lens, dev)
    start = _row_start(row_start, rows, seqs, dev)
    if out is None:
        out, ldo, ldo_head = _new((rows, q_heads, dim), _BF16, q.device, stream), q_heads * dim, dim
    else:
        ldo, ldo_head = _heads(out, "out", dev, q_heads, dim)
        if out.shape[0] != rows:
            raise ValueError(f"out has {out.shape[0]} rows, expected {rows}")
        # tokens of heads, or heads of tokens: either way the inner run has to fit between two of the outer
        if rows and not (ldo >= (q_heads - 1) * ldo_head + dim or ldo_head >= (rows - 1) * ldo + dim and ldo >= dim):
            raise ValueError("out's rows overlap")
    if lse is not None:
        _on(lse, "lse", _F32, dev)
        _dense(lse, "lse")
        if lse.shape != (rows, q_heads):
            raise ValueError(f"lse must be {(rows, q_heads)}")
    need = _attention_workspace(rows, 0 if start is None else 1, seqs, q_heads, heads, dim, min(width * page, 0x7FFFFFFF))
    ws = _new((need,), _U8, q.device, stream) if need else None
    _call("clef_kv_attention", q.data_ptr(), ldq, ldq_head, rows, start, q_heads, 0 if codes.dtype is _I8 else 1, c, pc, sc, ps,
          pages, heads, page, dim, table.data_ptr(), ldt, seqs, width, lens.data_ptr(),
          dim ** -0.5 if scale is None else float(scale), 1 if causal else 0, out.data_ptr(), ldo, ldo_head,
          None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(), need, _handle(dev, stream))
    return out


# ---------------------------------------------------------------- pages

def kv_reserve(table, lens, refs, grow, page: int, stream=None) -> None:
    """lens += grow (int32 [sequences]), with the pages of `page` tokens that
    takes: the lowest free ones, in the order of the sequences.  Changes
    nothing if the pool has too few (CLEF_ERR_NO_PAGES from poll_status)."""
    dev = _on(table, "table", _I32)
    ldt, seqs, width = _table(table, lens, dev)
    refs_at, grow_at = _ints(refs, "refs", dev), _ints(grow, "grow", dev, seqs)
    _call("clef_kv_reserve", table.data_ptr(), ldt, seqs, width, lens.data_ptr(), refs_at, refs.shape[0], int(page), grow_at,
          _handle(dev, stream))


def kv_fork(codes, scales, table, lens, refs, src, dst, stream=None) -> None:
    """Sequence dst[i] (empty before) becomes a copy of src[i]: whole pages are
    shared, a part-filled last page is copied to the lowest free page.  Changes
    nothing if the pool has too few free pages."""
    pool, dev = _pool(codes, scales)
    ldt, seqs, width = _table(table, lens, dev)
    refs_at, src_at = _ints(refs, "refs", dev, pool[5]), _ints(src, "src", dev)
    n = src.shape[0]
    dst_at = _ints(dst, "dst", dev, n)
    scratch = _new((2 * n,), _I32, table.device, stream)
    _call("clef_kv_fork", *pool, table.data_ptr(), ldt, seqs, width, lens.data_ptr(), refs_at, src_at, dst_at, n,
          scratch.data_ptr(), _handle(dev, stream))


def kv_free(table, lens, refs, seqs, page: int, stream=None) -> None:
    """The sequences listed in `seqs` (int32) give back their pages of `page`
    tokens and become empty."""
    dev = _on(table, "table", _I32)
    ldt, count, width = _table(table, lens, dev)
    refs_at, list_at = _ints(refs, "refs", dev), _ints(seqs, "seqs", dev)
    _call("clef_kv_free", table.data_ptr(), ldt, count, width, lens.data_ptr(), refs_at, refs.shape[0], int(page), list_at,
          seqs.shape[0], _handle(dev, stream))


def kv_compact(codes, scales, table, lens, refs, table_out=None, refs_out=None, stream=None):
    """Moves the held pages together at the pool's start and rewrites every
    sequence's row into table_out and refs into refs_out (in place where not
    given).  Returns the number of held pages, an int32 tensor of one value."""
    pool, dev = _pool(codes, scales)
    ldt, seqs, width = _table(table, lens, dev)
    table_out = table if table_out is None else table_out
    refs_out = refs if refs_out is None else refs_out
    pages = pool[5]
    refs_at, refs_out_at = _ints(refs, "refs", dev, pages), _ints(refs_out, "refs_out", dev, pages)
    ldt_out, s_out, w_out = _table(table_out, None, dev)
    if (s_out, w_out) != (seqs, width):
        raise ValueError("table_out has another shape than table")
    live = _new((1,), _I32, table.device, stream)
    scratch = _new((3 * pages + 1,), _I32, table.device, stream)
    if pages == 0:
        live.zero_()
    _call("clef_kv_compact", *pool, table.data_ptr(), ldt, seqs, width, lens.data_ptr(), refs_at, table_out.data_ptr(), ldt_out,
          refs_out_at, live.data_ptr(), scratch.data_ptr(), _handle(dev, stream))
    return live


def kv_copy_pages(codes, scales, src, dst, stream=None) -> None:
    """Page dst[i] becomes a copy of page src[i] (int32) in every plane; no
    target may also be a source or listed twice."""
    pool, dev = _pool(codes, scales)
    src_at = _ints(src, "src", dev)
    dst_at = _ints(dst, "dst", dev, src.shape[0])
    _call("clef_kv_copy_pages", *pool, src_at, dst_at, src.shape[0], _handle(dev, stream))
