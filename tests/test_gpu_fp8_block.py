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


def test_scales_of_each_block():
    """One block of K at a time, all others' scales zero: that block's sums, exactly its own scale."""
    m, n, k = 20, 264, 1040
    qx, sx, qw, sw, _ = inputs(m, n, k, 1)
    for rows in (m, 300):
        qx, sx = codes(rows, k, 5), torch.rand((rows, 9), generator=torch.Generator().manual_seed(6)).cuda() + 0.5
        for b in (0, 4, 8):
            only = torch.zeros_like(sx)
            only[:, b] = sx[:, b]
            check_linear(clef.fp8_block_linear(qx, only, qw, sw), (qx, only, qw, sw, None))


@pytest.mark.parametrize("m", [3, 40, 300])
def test_output_pitch_and_views(m):
    args = inputs(m, 136, 528, 7, with_bias=True)
    want = clef.fp8_block_linear(*args)
    out = torch.full((m, 400), 3.0, dtype=torch.bfloat16, device="cuda")
    got = clef.fp8_block_linear(*args, y=out[:, 8:144])
    assert torch.equal(got, want) and (out[:, :8] == 3).all() and (out[:, 144:] == 3).all()
    assert torch.equal(clef.fp8_block_linear(args[0].view(torch.float8_e4m3fn), args[1], args[2].view(torch.float8_e4m3fn), *args[3:]), want)
    wide = torch.full((m + 300, 136), 5.0, dtype=torch.bfloat16, device="cuda")     # rows behind the last are left alone
    clef.fp8_block_linear(*args, y=wide[:m])
    assert torch.equal(wide[:m], want) and (wide[m:] == 5).all()


@pytest.mark.parametrize("m", [5, 300])
def test_rows_of_nan_and_infinity_stay_theirs(m):
    args = list(inputs(m, 264, 528, 8))
    want = clef.fp8_block_linear(*args)
    args[0][2, 77] = 0x7F                       # the code that is no number
    args[1][4, 1] = float("inf")
    y = clef.fp8_block_linear(*args)
    keep = [i for i in range(m) if i not in (2, 4)]
    assert torch.equal(y[keep], want[keep]) and y[2].isnan().all() and not y[4].isfinite().any()


def test_empty():
    args = inputs(4, 128, 256, 9)
    y = clef.fp8_block_linear(args[0][:0], args[1][:0], *args[2:])
    assert y.shape == (0, 128)


@pytest.mark.parametrize("m", [1, 17, 50, 128, 300, 2000])
def test_same_bits_again_and_under_a_budget(m):
    """Repeated calls, calls on fewer SMs; with and without programmatic launches."""
    args = inputs(m, 1160, 2064, 10, with_bias=True)
    gu = inputs(m, 640, 1040, 11, gateup=True)
    want, h = clef.fp8_block_linear(*args), clef.fp8_block_gateup_swiglu(*gu)
    check_linear(want, args)
    check_gateup(h, gu)
    for _ in range(5):
        assert torch.equal(clef.fp8_block_linear(*args), want) and torch.equal(clef.fp8_block_gateup_swiglu(*gu), h)
    clef.set_pdl(False)
    try:
        assert torch.equal(clef.fp8_block_linear(*args), want)
    finally:
        clef.set_pdl(True)
    for sms in (2, 6, 100):
        clef.set_sm_budget(sms)
        try:
            assert torch.equal(clef.fp8_block_linear(*args), want) and torch.equal(clef.fp8_block_gateup_swiglu(*gu), h)
        finally:
            clef.set_sm_budget(0)
    assert clef.poll_status() == 0


def test_streams_and_graph():
    args, gu = inputs(40, 512, 1024, 12), inputs(300, 256, 1024, 13, gateup=True)
    want, h = clef.fp8_block_linear(*args), clef.fp8_block_gateup_swiglu(*gu)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    a = [clef.fp8_block_linear(*args, stream=s) for _ in range(4)]
    b = [clef.fp8_block_gateup_swiglu(*gu, stream=t) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in a) and all(torch.equal(x, h) for x in b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = clef.fp8_block_linear(*args)
    args[0].copy_(codes(40, 1024, 14))
    graph.replay()
    check_linear(y, args)


def test_captured_before_any_call():
    """In a process of its own: the first calls of each kind are recorded, not run."""
    import subprocess
    import sys
    code = """
import torch, w8a8_quantized_projections_gb300 as clef
x = {m: torch.randn(m, 512, device="cuda").to(torch.bfloat16) for m in (1, 30, 60, 120, 600, 2000)}
w = torch.randn(256, 512, device="cuda").to(torch.bfloat16)
n, pos, turns = w[0].contiguous(), torch.arange(2000, dtype=torch.int32, device="cuda"), clef.rotary_turns(64)
def run():
    qw, sw = clef.quant_fp8_block(w, 128)
    out = []
    for m, a in x.items():
        q, s = clef.rms_norm_quant(a, n, "fp8_b128")
        y = clef.fp8_block_linear(q, s, qw, sw)
        out += [y, clef.fp8_block_gateup_swiglu(q, s, qw, sw), clef.rotary(y.view(m, 4, 64), pos[:m], turns)]
    return out
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
assert all(torch.equal(a, b) for a, b in zip(got, run())) and clef.poll_status() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("m", [4, 300])
def test_a_wait_that_runs_out(m):
    """The issuer waits on what nothing signals: the status says so, and later calls are right."""
    args = inputs(m, 512, 1024, 15)
    want = clef.fp8_block_linear(*args)
    assert clef.poll_status() == 0
    clef.set_wait_limit_ns(20_000_000)
    clef.test_force_timeout(True)
    try:
        clef.fp8_block_linear(*args)
        assert clef.poll_status() == 4
    finally:
        clef.test_force_timeout(False)
        clef.set_wait_limit_ns(1_000_000_000)
    assert torch.equal(clef.fp8_block_linear(*args), want) and clef.poll_status() == 0


def test_far_rows():
    """Rows of the output past 2^32 bytes, and codes too."""
    if torch.cuda.mem_get_info()[0] < 24 * 2 ** 30:
        pytest.skip("memory")
    args = inputs(300, 128, 256, 16)
    pitch = 2 ** 24 + 64
    y = torch.empty(299 * pitch + 128, dtype=torch.bfloat16, device="cuda").as_strided((300, 128), (pitch, 1))
    assert torch.equal(clef.fp8_block_linear(*args, y=y), clef.fp8_block_linear(*args))
    del y
    m, k = 70000, 65536                         # 4.6 GB of codes
    qx = torch.zeros((m, k), dtype=torch.uint8, device="cuda")
    sx = torch.zeros((m, 512), device="cuda")
    last = inputs(16, 128, k, 17)
    qx[-16:], sx[-16:] = last[0], last[1]
    y = clef.fp8_block_linear(qx, sx, *last[2:])
    check_linear(y[-16:], last)
    assert not y[:-16].any()


def test_refusals():
    qx, sx, qw, sw, _ = inputs(4, 256, 512, 18)
    for call in (lambda: clef.fp8_block_linear(qx, sx[:, :3], qw, sw), lambda: clef.fp8_block_linear(qx, sx, qw, sw[:1]),
                 lambda: clef.fp8_block_linear(qx, sx[:3], qw, sw), lambda: clef.fp8_block_linear(qx[:, :256], sx, qw, sw),
                 lambda: clef.fp8_block_linear(qx.view(torch.int8), sx, qw, sw), lambda: clef.fp8_block_linear(qx, sx.double(), qw, sw),
                 lambda: clef.fp8_block_linear(qx, sx, qw, sw, torch.zeros(255, dtype=torch.bfloat16, device="cuda")),
                 lambda: clef.fp8_block_linear(qx, sx, qw, sw, y=torch.zeros((4, 255), dtype=torch.bfloat16, device="cuda")),
                 lambda: clef.fp8_block_linear(qx.cpu(), sx, qw, sw), lambda: clef.fp8_block_linear(qx[0], sx, qw, sw),
                 lambda: clef.fp8_block_gateup_swiglu(qx, sx, qw[:255].contiguous(), sw)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: clef.fp8_block_linear(qx, sx, qw[:252].contiguous(), sw),
                 lambda: clef.fp8_block_gateup_swiglu(qx, sx, qw[:240].contiguous(), sw),
                 lambda: clef.fp8_block_linear(*inputs(4, 128, 24, 19))):
        with pytest.raises(clef.ClefError) as e:
            call()
        assert e.value.status == 1
