"""64-bit models of the operators between the projections, for the tests."""
from __future__ import annotations

import math

import numpy as np
import torch

TOP = {"int8_h128": 127.0, "fp8": 448.0, "fp8_h128": 448.0, "fp8_b128": 448.0}
U = 2.0 ** -24                      # half a step of fp32, relative


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


def e4m3(t: torch.Tensor) -> np.ndarray:
    return t.detach().view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)


def hadamard() -> np.ndarray:
    i = np.arange(128)
    odd = np.array([[bin(a & b).count("1") & 1 for b in i] for a in i])
    return (1.0 - 2.0 * odd) / math.sqrt(128.0)


def rotated(v: np.ndarray) -> np.ndarray:
    return (v.reshape(-1, 128) @ hadamard()).reshape(v.shape)


def bf16_off(ref: np.ndarray) -> np.ndarray:
    """Half a bf16 step: 2^-8 of the value, or half the smallest subnormal."""
    return np.abs(ref) * 2.0 ** -8 + 2.0 ** -134


def norm(x, w, eps, residual=None):
    h = f64(x) + (0.0 if residual is None else f64(residual))
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * f64(w)


def norm_rel(K: int) -> float:
    """fp32 error of a normed value, relative.  The sum h (1 U), the sum of squares: 64 products a thread in
    a row at most, then ten halvings, each fused or added once: 74 U, of which the root takes half; mean,
    eps, root and its rounding 4 U; two products 2 U."""
    return (1 + 74 + 37 + 4 + 2) * U


def blocks_of(v: np.ndarray) -> np.ndarray:
    """[rows][blocks][128], short last blocks filled with zeros."""
    m, k = v.shape
    b = -(-k // 128)
    out = np.zeros((m, b * 128))
    out[:, :k] = v
    return out.reshape(m, b, 128)


def block_amax(v: np.ndarray, rows: int) -> np.ndarray:
    a = np.abs(blocks_of(v)).max(-1)
    return np.stack([a[i:i + rows].max(0) for i in range(0, a.shape[0], rows)]) if a.shape[0] else a


def spread(s: np.ndarray, rows: int, shape) -> np.ndarray:
    return np.repeat(np.repeat(s, rows, 0)[: shape[0]], 128, 1)[:, : shape[1]]


def check_codes(got, scale, v, amax, top, err):
    """Codes `got` (values of codes) with scales (spread over the elements) stand for v within half a code
    step and `err` of the value's own computation."""
    step = 0.5 * scale if top == 127.0 else np.maximum(np.abs(v) / 16, 2.0 ** -10 * scale)
    # the scale and its reciprocal are rounded once each, the product once
    off = step * (1 + 2.0 ** -20) + err + 4 * U * np.abs(v)
    assert (np.abs(got * scale - v) <= off).all(), float((np.abs(got * scale - v) - off).max())
    assert (np.abs(got) <= top).all()
    assert (np.abs(scale - amax / top) <= (amax / top) * 4 * U + err / top + 2.0 ** -149).all()


def rotary(x, pos, turns, gain, interleaved):
    """In 64 bits from exact whole-number angles: (values, fp32 bound)."""
    rot = 2 * len(turns)
    y = f64(x)
    first = np.arange(rot // 2) * (2 if interleaved else 1)
    second = first + (1 if interleaved else rot // 2)
    p = [int(t) for t in pos]
    q = [int(t) for t in turns]
    frac = np.array([[((a * b + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 64 for b in q] for a in p]).reshape(len(p), len(q))
    c, s = np.cos(2 * np.pi * frac)[:, None], np.sin(2 * np.pi * frac)[:, None]
    a, b = y[..., first], y[..., second]
    off = np.zeros_like(y)
    # an angle is rounded to fp32 (at most pi 2^-24) and cut at 2^-32 turns, cosine and sine are off by two
    # units of 2^-24 and their products with gain by one, the rotation by two more
    off[..., first] = off[..., second] = 10 * U * abs(gain) * (np.abs(a) + np.abs(b))
    y[..., first], y[..., second] = gain * (a * c - b * s), gain * (b * c + a * s)
    return y, off
