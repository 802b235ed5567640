"""The 4-bit linear and its packing against 64-bit models: odd sizes, every
group length, one to many rows, pitches, a row's bits independent of M, and
refusals.

Tolerance of y: one bf16 ulp (its rounding, and a neighbour where the fp32 sum
differs) plus (K / 16 + 2) 2^-23 sum |s c x|, the bound on fp32 sums in
16-deep steps."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from decode_util import bf16, bf16_ulp, dev_bf16, w4_codes, w4_pack

pytestmark = pytest.mark.gpu


def check(x, codes, sw, group, bias, got):
    s = np.repeat(sw.astype(np.float64), group, 1)[:, : codes.shape[1]]
    w = codes * s
    ref = x.astype(np.float64) @ w.T + (0 if bias is None else bias.astype(np.float64))
    mag = np.abs(x.astype(np.float64)) @ np.abs(w).T + (0 if bias is None else np.abs(bias))
    tol = bf16_ulp(ref) + (x.shape[1] / 16 + 2) * 2.0 ** -23 * mag
    d = np.abs(got.astype(np.float64) - ref)
    assert (d <= tol).all(), f"{(d > tol).sum()} of {d.size} outside, worst {(d / tol).max():.2f} of the bound"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K,bias", [
    (1, 128, 128, False), (1, 1, 8, True), (2, 7, 136, True), (3, 129, 256, False), (8, 300, 1000, True),
    (9, 257, 1152, False), (13, 1025, 520, True), (16, 64, 4096, False), (17, 130, 264, True), (40, 250, 2056, False),
    (1, 5120, 6144, False), (5, 2048, 17408, True), (12, 48, 65536, False), (16, 100, 17408, True), (1, 20000, 128, False),
])
def test_linear(M, N, K, bias, group):
    rng = np.random.default_rng(M * 7 + N + K + group)
    x = bf16(rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 20, 1))
    codes = rng.integers(-8, 8, (N, K))
    kp = (K + 127) // 128 * 128
    sw = bf16(rng.uniform(0.001, 0.05, (N, kp // group)))
    b = bf16(rng.standard_normal(N)) if bias else None
    y = clef.w4_linear(dev_bf16(x), torch.from_numpy(w4_pack(codes)).cuda(), dev_bf16(sw),
                       None if b is None else dev_bf16(b))
    check(x, codes, sw, group, b, y.float().cpu().numpy())
    assert clef.poll_status() == 0


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 8), (5, 136), (64, 128), (33, 4104)])
def test_pack(N, K, group):
    """s = bf16(amax / 7) and c = rne(w / s), in IEEE fp32; weights past K are zeros."""
    rng = np.random.default_rng(N + K)
    w = bf16(rng.standard_normal((N, K)) * 0.02)
    w[N // 2] = 0
    qw, sw = clef.quant_w4(dev_bf16(w), group)
    kp = (K + 127) // 128 * 128
    full = np.zeros((N, kp), np.float32)
    full[:, :K] = w
    s = bf16(np.abs(full.reshape(N, -1, group)).max(-1) / np.float32(7))
    rep = np.repeat(s, group, 1)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(rep > 0, np.clip(np.rint(full / rep), -8, 7), 0).astype(np.int64)
    assert np.array_equal(sw.float().cpu().numpy(), s)
    assert np.array_equal(w4_codes(qw.cpu().numpy(), kp), c)
    # the packed weights multiply as the weights they stand for
    x = bf16(rng.standard_normal((2, K)))
    check(x, c[:, :K], s, group, None, clef.w4_linear(dev_bf16(x), qw, sw).float().cpu().numpy())


@pytest.mark.parametrize("group", [32, 64, 128])
def test_rows_do_not_depend_on_m(group):
    """The bits of a row are the same alone, among others and at an output pitch."""
    rng = np.random.default_rng(5)
    x = dev_bf16(rng.standard_normal((37, 2176)))
    qw, sw = clef.quant_w4(dev_bf16(rng.standard_normal((515, 2176)) * 0.02), group)
    whole = clef.w4_linear(x, qw, sw)
    for a, b in ((0, 1), (1, 3), (3, 11), (11, 24), (24, 37)):
        assert torch.equal(clef.w4_linear(x[a:b], qw, sw), whole[a:b])
    wide = torch.zeros((37, 517), dtype=torch.bfloat16, device="cuda")       # odd pitch, 2-byte aligned rows
    out = wide[:, 1:516]
    clef.w4_linear(x, qw, sw, y=out)
    assert torch.equal(out, whole) and not wide[:, 0].any() and not wide[:, 516].any()
    xw = torch.zeros((37, 2200), dtype=torch.bfloat16, device="cuda")
    xw[:, 8:2184] = x
    assert torch.equal(clef.w4_linear(xw[:, 8:2184], qw, sw), whole)


def test_streams_and_graph():
    """A call on a side stream orders with its producer there, and replays from a graph."""
    rng = np.random.default_rng(6)
    qw, sw = clef.quant_w4(dev_bf16(rng.standard_normal((640, 1024)) * 0.02))
    x = dev_bf16(rng.standard_normal((4, 1024)))
    ref = clef.w4_linear(x, qw, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = clef.w4_linear(x, qw, sw, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clef.w4_linear(x, qw, sw, y=out)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, clef.w4_linear(x, qw, sw))


def test_refusals():
    x = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda")
    qw = torch.zeros((64, 128), dtype=torch.uint8, device="cuda")
    sw = torch.zeros((64, 2), dtype=torch.bfloat16, device="cuda")
    clef.w4_linear(x, qw, sw)
    assert clef.w4_linear(x[:0], qw, sw).shape == (0, 64)
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(qw=qw[:, :64]), dict(sw=sw[:-1]), dict(sw=sw[:, :0]),
                dict(sw=torch.zeros((64, 3), dtype=torch.bfloat16, device="cuda")), dict(qw=qw.cpu()),
                dict(bias=torch.zeros(63, dtype=torch.bfloat16, device="cuda")),
                dict(y=torch.zeros((2, 63), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            clef.w4_linear(**{**dict(x=x, qw=qw, sw=sw), **bad})
    with pytest.raises(clef.ClefError):
        clef.w4_linear(torch.zeros((2, 260), dtype=torch.bfloat16, device="cuda")[:, 1:257], qw, sw)   # misaligned rows
    with pytest.raises(ValueError):
        clef.quant_w4(x, 48)
    with pytest.raises(clef.ClefError):
        clef.quant_w4(torch.zeros((2, 20), dtype=torch.bfloat16, device="cuda"))                         # K % 8
    assert clef.poll_status() == 0


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(13, 5000, 17408), (16, 5120, 17408), (9, 9001, 6144), (12, 8200, 9000)])
def test_many_tiles(M, N, K, group):
    """More tiles than CTAs: the bits of single rows, and 64-bit sums for the first and last weight rows."""
    g = torch.Generator(device="cuda").manual_seed(M + N + group)
    kp = (K + 127) // 128 * 128
    qw = torch.randint(0, 256, (N, kp // 2), generator=g, device="cuda", dtype=torch.uint8)
    if kp > K:      # the padding's codes are those of zero; K is a multiple of 8, so whole bytes belong to it
        zeros = np.zeros((1, kp), np.int64)
        mask = w4_pack(np.where(np.arange(kp) < K, 7, -8)[None]) == 0xFF
        qw = torch.where(torch.from_numpy(mask).cuda(), qw, torch.from_numpy(w4_pack(zeros)).cuda())
    sw = (torch.rand((N, kp // group), generator=g, device="cuda") * 0.05 + 0.001).to(torch.bfloat16)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    y = clef.w4_linear(x, qw, sw)
    for m in (0, M // 2, M - 1):
        assert torch.equal(clef.w4_linear(x[m:m + 1], qw, sw)[0], y[m])
    for rows in (slice(0, 40), slice(N - 40, N)):
        check(x.float().cpu().numpy(), w4_codes(qw[rows].cpu().numpy(), K), sw[rows].float().cpu().numpy(), group, None,
              y[:, rows].float().cpu().numpy())
    assert clef.poll_status() == 0


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 40, 256), (5, 130, 2056), (9, 300, 1152), (16, 100, 4096)])
def test_magnitudes(M, N, K, group):
    """Rows of x from bf16's smallest normal numbers to its largest."""
    rng = np.random.default_rng(M + N + K + group)
    amp = np.asarray([3e38, 1.0, 2.0 ** 116, 2.0 ** 113, 2.0 ** 120, 1e-37, 1e20, 2.0 ** 127])[np.arange(M) % 8][:, None]
    x = bf16(rng.uniform(-1, 1, (M, K)) * amp)
    codes = rng.integers(-8, 8, (N, K))
    kp = (K + 127) // 128 * 128
    sw = bf16(rng.uniform(1e-6, 2e-5, (N, kp // group)))
    b = bf16(rng.standard_normal(N))
    qw = torch.from_numpy(w4_pack(codes)).cuda()
    y = clef.w4_linear(dev_bf16(x), qw, dev_bf16(sw), dev_bf16(b))
    check(x, codes, sw, group, b, y.float().cpu().numpy())
    for m in range(M):
        assert torch.equal(clef.w4_linear(dev_bf16(x[m:m + 1]), qw, dev_bf16(sw), dev_bf16(b))[0], y[m])
    if M > 1:      # what is not finite stays in its row
        for bad in (np.inf, -np.inf, np.nan):
            w = x.copy()
            w[1, 7] = bad
            z = clef.w4_linear(dev_bf16(w), qw, dev_bf16(sw), dev_bf16(b))
            assert z[1].isnan().all()
            z[1] = y[1]
            assert torch.equal(z, y)
    assert clef.poll_status() == 0


def test_most_rows():
    """The most rows that are allowed, over a K whose blocks have eight rows: more blocks than a grid has."""
    M, N, K = 1 << 19, 24, 29952
    rng = np.random.default_rng(7)
    qw, sw = clef.quant_w4(dev_bf16(rng.standard_normal((N, K)) * 0.02), 128)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    few = dev_bf16(rng.standard_normal((21, K)))
    ref = clef.w4_linear(few, qw, sw)
    at = torch.tensor([*range(8), M // 2, *range(65535 * 8 - 4, M)], device="cuda")
    x[at] = few
    y = torch.full((M, N + 2), 3.0, dtype=torch.bfloat16, device="cuda")
    clef.w4_linear(x, qw, sw, y=y[:, :N])
    assert torch.equal(y[at, :N], ref) and (y[:, N:] == 3).all()
    y[at] = 0
    assert not y[:, :N].any()
    assert clef.poll_status() == 0
