"""Linears over e4m3 codes in blocks of 128 against 64-bit sums of the same codes."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from between_util import U, bf16_off, e4m3, f64, spread

pytestmark = pytest.mark.gpu


def codes(m, k, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((m, k), generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).cuda()


def scales(m, k, seed, low=-6, high=6):
    """Powers of two to the low .. high times 1 .. 2, some of them zeros."""
    g = torch.Generator().manual_seed(seed)
    b = -(-k // 128)
    s = torch.exp2(torch.randint(low, high, (m, b), generator=g).float()) * (1 + torch.rand((m, b), generator=g))
    s[torch.rand((m, b), generator=g) < 0.05] = 0
    return (s / 500).cuda()


def inputs(m, n, k, seed, with_bias=False, gateup=False):
    rows = 2 * n if gateup else n
    bias = torch.randn(rows, generator=torch.Generator().manual_seed(seed + 4)).to(torch.bfloat16).cuda() if with_bias else None
    return codes(m, k, seed), scales(m, k, seed + 1), codes(rows, k, seed + 2), scales(-(-rows // 128), k, seed + 3, -3, 3) / 8, bias


def product(qx, sx, qw, sw, bias):
    """The sums in 64 bits, and how far fp32 ones may be off: in each block of 128 the products are added in
    at most sixteen steps, each off by a unit of 2^-23 of what the block's products add up to at most; a
    scale is one product, a block one addition to the total, and the bias one."""
    x, w = e4m3(qx) * spread(f64(sx), 1, qx.shape), e4m3(qw) * spread(f64(sw), 128, qw.shape)
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    off = (2 * 16 + 2 + sx.shape[1] + 2) * U * mag
    if bias is not None:
        y = y + f64(bias)
        off = off + 2 * U * np.abs(f64(bias))
    return y, off


def check_linear(y, args):
    ref, off = product(*args)
    assert (np.abs(f64(y) - ref) <= off + bf16_off(ref) * (1 + 2.0 ** -8)).all(), float(np.abs(f64(y) - ref).max())


def check_gateup(h, args):
    y, off = product(*args)
    n = y.shape[1] // 2
    g, u, dg, du = y[:, :n], y[:, n:], off[:, :n], off[:, n:]
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    ref = silu * u
    # silu's slope is at most 1.1; exp, sum, quotient and product are a few units each
    err = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + (12 + np.abs(g)) * U * np.abs(ref) + 2.0 ** -120
    assert (np.abs(f64(h) - ref) <= err + bf16_off(ref) * (1 + 2.0 ** -8)).all()


FEW = [1, 2, 13, 16, 17, 31, 33, 64, 65, 100, 128]
SHAPES = [(8, 16), (24, 128), (136, 144), (128, 256), (264, 1040), (520, 2048), (2048, 528), (64, 4112)]


@pytest.mark.parametrize("m", FEW)
@pytest.mark.parametrize("n,k", SHAPES)
def test_few_rows(m, n, k):
    args = inputs(m, n, k, m + n + k, with_bias=(m + n) % 3 == 0)
    check_linear(clef.fp8_block_linear(*args), args)
    assert clef.poll_status() == 0


@pytest.mark.parametrize("m", [129, 256, 257, 300, 511, 1500])
@pytest.mark.parametrize("n,k", SHAPES)
def test_many_rows(m, n, k):
    args = inputs(m, n, k, m + n + k, with_bias=(m + n) % 3 == 0)
    check_linear(clef.fp8_block_linear(*args), args)
    assert clef.poll_status() == 0


@pytest.mark.parametrize("m", FEW + [129, 256, 300, 770])
@pytest.mark.parametrize("n,k", [(128, 16), (128, 384), (384, 1040), (2176, 272), (256, 4112)])
def test_gateup(m, n, k):
    args = inputs(m, n, k, m + n + k, with_bias=(m + n // 128) % 2 == 0, gateup=True)
    check_gateup(clef.fp8_block_gateup_swiglu(*args), args)
    assert clef.poll_status() == 0
