"""Bindings for what stands between a layer's projections: the norm with the residual's
addition and 8-bit outputs, rotary positions, and the linears over e4m3 codes with a
scale for each block of 128.

Arguments are checked and marshalled by the compiled module of ``decode.py``; what each
call computes is in ``include/clef.h``.
"""
from __future__ import annotations

import math

import torch

from . import decode as _decode

__all__ = ["rms_norm", "rms_norm_quant", "quant_fp8_block", "fp8_block_linear", "fp8_block_gateup_swiglu", "rotary", "rotary_turns"]

NORM_MODES = {"int8_h128": 0, "fp8": 1, "fp8_h128": 2, "fp8_b128": 3}


def _ext():
    return _decode._ext or _decode._load()


# ---------------------------------------------------------------- norms

def rms_norm(x, w, eps: float = 1e-6, residual=None, residual_out=None, y=None, stream=None):
    """bf16(h w / sqrt(mean(h^2) + eps)) of the rows of h = x + residual (bf16 [M][K]; x alone
    without one).  bf16(h) goes to residual_out, or to residual itself where it is not given.
    y may be x itself."""
    return _ext().rms_norm(x, w, eps, residual, residual_out, y, stream)


def rms_norm_quant(x, w, mode: str = "int8_h128", eps: float = 1e-6, residual=None, residual_out=None, y=None, q=None,
                   scale=None, stream=None):
    """The norm's 8-bit codes and scales, as the linears take them: modes "int8_h128", "fp8" and
    "fp8_h128" a scale a row, "fp8_b128" a scale for each 128 values of a row (fp8_block_linear).
    Codes are those of the unrounded fp32 result.  y (bf16 [M][K], optional) also receives the
    result itself.  Returns (q [M][K], scale fp32 [M] or [M][ceil(K / 128)])."""
    return _ext().rms_norm_quant(x, w, NORM_MODES[mode], eps, residual, residual_out, y, q, scale, stream)


# ---------------------------------------------------------------- blocks of 128

def quant_fp8_block(x, rows: int = 1, q=None, scale=None, stream=None):
    """e4m3 codes of bf16 x [M][K] with a scale for each block of `rows` (1 for activations, 128
    for weights) by 128: (q uint8 [M][K], scale fp32 [ceil(M / rows)][ceil(K / 128)])."""
    return _ext().quant_fp8_block(x, rows, q, scale, stream)


def fp8_block_linear(qx, sx, qw, sw, bias=None, y=None, stream=None):
    """y = bf16(x W^T + bias) for e4m3 codes in blocks: qx [M][K] with sx [M][ceil(K / 128)], qw [N][K]
    with sw [ceil(N / 128)][ceil(K / 128)] (quant_fp8_block with rows = 1 and 128, rms_norm_quant)."""
    return _ext().fp8_block(qx, sx, qw, sw, bias, y, stream, False)


def fp8_block_gateup_swiglu(qx, sx, qw_gu, sw_gu, bias_gu=None, h=None, stream=None):
    """h = bf16(silu(g) * u) for packed gate/up codes in blocks, [2N][K] with N a multiple of 128."""
    return _ext().fp8_block(qx, sx, qw_gu, sw_gu, bias_gu, h, stream, True)


# ---------------------------------------------------------------- rotary positions

def rotary_turns(rot: int, theta: float = 10000.0, scaling: str | None = None, factor: float = 1.0, original: int = 4096,
                 slow: float = 1.0, fast: float = 32.0, device="cuda") -> torch.Tensor:
    """The table that rotary() takes for heads of which `rot` values are rotated: int64 [rot / 2],
    the turns a position of frequencies theta ** (-2 i / rot), in units of 2^-64, modulo one turn.

    scaling, for contexts `factor` times as long as the `original` ones:
      None        the frequencies as they are;
      "linear"    all divided by factor;
      "theta"     theta times factor ** (rot / (rot - 2)): the slowest divided by factor, the fastest kept;
      "by_parts"  those with `fast` turns or more in `original` positions kept, those with `slow` or
                  fewer divided by factor, between the two mixed in proportion to their turns.
    Make it once and keep it: it is built on the host and copied."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, not {rot}")
    if scaling not in (None, "linear", "theta", "by_parts"):
        raise ValueError(f"scaling {scaling!r}: None, linear, theta or by_parts")
    if not (0.0 < theta < math.inf and 1.0 <= factor < math.inf and original > 0 and 0.0 <= slow < fast):
        raise ValueError("theta and original must be positive, factor at least 1, slow below fast")
    if scaling == "theta":
        if rot == 2:
            raise ValueError("scaling by theta needs more than one frequency")
        theta = theta * factor ** (rot / (rot - 2))
    table = []
    for i in range(rot // 2):
        turns = theta ** (-2.0 * i / rot) / (2.0 * math.pi)
        if scaling == "linear":
            turns /= factor
        elif scaling == "by_parts":
            keep = min(1.0, max(0.0, (turns * original - slow) / (fast - slow)))
            turns = turns * keep + turns / factor * (1.0 - keep)
        u = round(turns * 2.0 ** 64) % 2 ** 64
        table.append(u - 2 ** 64 if u >= 2 ** 63 else u)
    return torch.tensor(table, dtype=torch.int64, device=device)


def rotary(x, pos, turns, gain: float = 1.0, interleaved: bool = False, out=None, stream=None):
    """Heads of x (bf16 [tokens][heads][dim]) rotated by their tokens' positions (int32 [tokens]):
    pairs (i, i + rot / 2), or (2 i, 2 i + 1) where interleaved, of the first rot = 2 len(turns)
    values of a head, times gain; the others are copied.  turns: a table of rotary_turns.
    out may be x itself."""
    return _ext().rotary(x, pos, turns, gain, interleaved, out, stream)
