"""The norm with the residual's addition, its codes, and the quantizer of blocks of 128, against 64 bits."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from between_util import (TOP, U, bf16_off, block_amax, check_codes, e4m3, f64, norm, norm_rel, rotated, spread)

pytestmark = pytest.mark.gpu
MODES = ["int8_h128", "fp8", "fp8_h128", "fp8_b128"]
# (rows, columns): lanes of a warp a row (to 512), a CTA a row (to 16,384), four chunks a thread beyond
SIZES = [(1, 16), (5, 112), (17, 128), (3, 144), (9, 256), (2, 272), (33, 512), (1, 528), (3, 640), (2, 4096), (1, 5120),
         (7, 5136), (2, 16384), (2, 16400), (1, 17408), (1, 32768)]


def values(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    if shape[-1] > 3:
        x[..., 3] *= 30
    return x.to(torch.bfloat16).cuda()


def weight(k, seed):
    return (1 + 0.3 * torch.randn(k, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).cuda()


def codes_and_scale(q, scale, mode, shape):
    got = q.cpu().numpy().astype(np.float64) if mode == "int8_h128" else e4m3(q)
    s = f64(scale)
    return got, spread(s, 1, shape) if mode == "fp8_b128" else np.broadcast_to(s[:, None], shape)


def check_quant(q, scale, mode, v, rel):
    """v: the normed rows in 64 bits, off by `rel` of themselves in the kernel."""
    err = rel * np.abs(v)
    if mode.endswith("h128"):
        # seven stages of the rotation, each rounded, of values up to the block's sum
        total = np.repeat(np.abs(v).reshape(-1, 128).sum(-1), 128).reshape(v.shape) / np.sqrt(128.0)
        err, v = (rel + 9 * U) * total, rotated(v)
    if mode == "fp8_b128":
        amax = spread(block_amax(v, 1), 1, v.shape)
        err = np.maximum(err, rel * amax)
    else:
        amax = np.broadcast_to(np.abs(v).max(-1, keepdims=True), v.shape)
        err = np.broadcast_to(np.maximum(err, rel * amax).max(-1, keepdims=True), v.shape)
    got, s = codes_and_scale(q, scale, mode, v.shape)
    check_codes(got, s, v, amax, TOP[mode], err)


@pytest.mark.parametrize("m,k", SIZES)
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm(m, k, with_residual):
    x, w, r = values((m, k), 1), weight(k, 2), values((m, k), 3) if with_residual else None
    ref = norm(x, w, 1e-6, r)
    out = None if r is None else torch.full_like(r, -1.0)
    y = clef.rms_norm(x, w, residual=r, residual_out=out)
    assert (np.abs(f64(y) - ref) <= bf16_off(ref) + norm_rel(k) * np.abs(ref)).all()
    if with_residual:
        total = (x.float() + r.float()).to(torch.bfloat16)
        assert torch.equal(out, total)
        again = r.clone()
        assert torch.equal(clef.rms_norm(x, w, residual=again), y) and torch.equal(again, total)      # in place
    assert clef.poll_status() == 0


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("m,k", SIZES)
def test_codes(mode, m, k):
    if mode.endswith("h128") and k % 128:
        pytest.skip("whole blocks are rotated")
    x, w, r = values((m, k), 4), weight(k, 5), values((m, k), 6)
    ref = norm(x, w, 1e-5, r)
    total, y = torch.empty_like(r), torch.empty_like(x)
    q, scale = clef.rms_norm_quant(x, w, mode, 1e-5, residual=r, residual_out=total, y=y)
    assert tuple(scale.shape) == ((m, -(-k // 128)) if mode == "fp8_b128" else (m,))
    check_quant(q, scale, mode, ref, norm_rel(k))
    assert torch.equal(total, (x.float() + r.float()).to(torch.bfloat16))
    assert torch.equal(y, clef.rms_norm(x, w, 1e-5, residual=r.clone()))
    q2, s2 = clef.rms_norm_quant(x, w, mode, 1e-5, residual=r.clone())             # without y: the same codes
    assert torch.equal(q2, q) and torch.equal(s2, scale)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("k", [128, 512, 2048])
def test_a_row_does_not_depend_on_the_others(mode, k):
    x, w, r = values((70, k), 7), weight(k, 8), values((70, k), 9)
    x[11] = float("nan")
    x[12] = 3e38
    r[12] = 0.0
    q, s = clef.rms_norm_quant(x, w, mode, residual=r.clone())
    y = clef.rms_norm(x, w, residual=r.clone())
    for i in (0, 10, 13, 69):
        qi, si = clef.rms_norm_quant(x[i:i + 1], w, mode, residual=r[i:i + 1].clone())
        assert torch.equal(qi[0], q[i]) and torch.equal(si[0], s[i])
        assert torch.equal(clef.rms_norm(x[i:i + 1], w, residual=r[i:i + 1].clone())[0], y[i])


@pytest.mark.parametrize("k", [128, 640, 5120, 20480])
@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** 100, 2.0 ** 125, 2.0 ** -30, 2.0 ** -70])
def test_values_of_any_size(k, size):
    """Squares past fp32, or below it; eps of its own size beside them."""
    x, w = values((3, k), 10), weight(k, 11)
    x[:, 3] /= 30
    x = (x.float() * size).to(torch.bfloat16)
    x[1] = values((1, k), 12)[0]                     # an ordinary row between them
    ref = norm(x, w, 1e-6)
    y = clef.rms_norm(x, w)
    # squares of 2^-140 are lost beside an eps of 1e-6
    assert (np.abs(f64(y) - ref) <= bf16_off(ref) + norm_rel(k) * np.abs(ref) + 2.0 ** -126).all()
    q, scale = clef.rms_norm_quant(x, w, "fp8_b128")
    check_quant(q, scale, "fp8_b128", ref, norm_rel(k))


@pytest.mark.parametrize("mode", MODES)
def test_zero_rows(mode):
    x, w = values((6, 384), 13), weight(384, 14)
    x[2] = 0
    x[4, 128:256] = 0
    q, scale = clef.rms_norm_quant(x, w, mode)
    assert not q[2].any() and not scale[2].any()
    if mode == "fp8_b128":
        assert not q[4, 128:256].any() and float(scale[4, 1]) == 0.0 and float(scale[4, 0]) > 0
    assert not clef.rms_norm(x, w)[2].any()


def test_strides_and_empty():
    wide = values((9, 5 * 640), 15)
    x, r = wide[:, 640:1280], wide[:, 1920:2560]
    w = weight(640, 16)
    out = torch.full((9, 3 * 640), 7.0, dtype=torch.bfloat16, device="cuda")
    total, y = out[:, :640], out[:, 1280:]
    q, scale = clef.rms_norm_quant(x, w, "int8_h128", residual=r, residual_out=total, y=y)
    dense = r.contiguous()
    q2, s2 = clef.rms_norm_quant(x.contiguous(), w, "int8_h128", residual=dense)
    assert torch.equal(q, q2) and torch.equal(scale, s2) and torch.equal(total, dense)
    assert (out[:, 640:1280] == 7.0).all()
    assert torch.equal(y, clef.rms_norm(x, w, residual=r, residual_out=torch.empty_like(dense)))
    e = torch.empty((0, 640), dtype=torch.bfloat16, device="cuda")
    assert clef.rms_norm(e, w, residual=e).shape == (0, 640)
    q, s = clef.rms_norm_quant(e, w, "fp8_b128")
    assert q.shape == (0, 640) and s.shape == (0, 5)
    x = values((4, 640), 17)
    assert torch.equal(clef.rms_norm(x.clone(), w), clef.rms_norm(x, w, y=x))     # over its input


# ---------------------------------------------------------------- blocks of 128

@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m,k", [(1, 16), (1, 128), (3, 144), (127, 240), (128, 256), (129, 2048), (300, 1040), (2, 65536)])
def test_quant_block(rows, m, k):
    wide = values((m, k + 8), 18)
    x = wide[:, :k]
    x[0, :16] = 0
    if k > 144:
        x[:, 128:256] = 0
    q, scale = clef.quant_fp8_block(x, rows)
    v = f64(x)
    s = f64(scale)
    assert s.shape == (-(-m // rows), -(-k // 128))
    amax = block_amax(v, rows)
    check_codes(e4m3(q), spread(s, rows, v.shape), v, spread(amax, rows, v.shape), 448.0, np.zeros_like(v))
    assert ((s == 0) == (amax == 0)).all()
    # the codes are exact: correctly rounded products with the rounded factor
    with np.errstate(divide="ignore", over="ignore"):
        r = np.where(amax > 0, np.minimum(np.float32(448) / amax.astype(np.float32), np.float32(3.4028235e38)), 0).astype(np.float32)
    want = torch.from_numpy(v.astype(np.float32) * spread(r, rows, v.shape).astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu(), want.view(torch.uint8))


def test_quant_block_many_rows():
    """More blocks than the CTAs of a call, and the smallest values."""
    x = values((70001, 144), 19)
    x[5] = 2.0 ** -133
    q, scale = clef.quant_fp8_block(x, 1)
    v = f64(x)
    amax = block_amax(v, 1)
    s = f64(scale)
    assert (np.abs(s - amax / 448) <= amax / 448 * 2 * U + 2.0 ** -149).all()
    keep = np.arange(70001) != 5
    check_codes(e4m3(q)[keep], spread(s, 1, v.shape)[keep], v[keep], spread(amax, 1, v.shape)[keep], 448.0, 0.0)
    assert np.isfinite(e4m3(q)).all()


def test_stream_and_graph():
    x, w, r = values((40, 1024), 20), weight(1024, 21), values((40, 1024), 22)
    want = clef.rms_norm_quant(x, w, "fp8_b128", residual=r.clone())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    total = torch.empty_like(r)
    got = clef.rms_norm_quant(x, w, "fp8_b128", residual=r, residual_out=total, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = clef.rms_norm_quant(x, w, "fp8_b128", residual=r, residual_out=total)
    for seed in (23, 24):
        x.copy_(values((40, 1024), seed))
        graph.replay()
        want = clef.rms_norm_quant(x, w, "fp8_b128", residual=r.clone())
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    x, w, r = values((4, 256), 25), weight(256, 26), values((4, 256), 27)
    for call in (lambda: clef.rms_norm(x, w[:128]), lambda: clef.rms_norm(x.float(), w), lambda: clef.rms_norm(x.cpu(), w),
                 lambda: clef.rms_norm(x, w, residual=r[:3]), lambda: clef.rms_norm(x, w, residual_out=r),
                 lambda: clef.rms_norm(x, w, y=r[:, :128]), lambda: clef.rms_norm(x.t(), w),
                 lambda: clef.rms_norm_quant(x, w, "fp8", q=torch.empty((4, 256), dtype=torch.int8, device="cuda")),
                 lambda: clef.rms_norm_quant(x, w, "fp8_b128", scale=torch.empty(4, device="cuda")),
                 lambda: clef.quant_fp8_block(x, 64), lambda: clef.quant_fp8_block(x, scale=torch.empty(3, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(KeyError):
        clef.rms_norm_quant(x, w, "int8")
    for call in (lambda: clef.rms_norm(x, w, 0.0), lambda: clef.rms_norm(x, w, float("nan")),
                 lambda: clef.rms_norm(x[:, :24], w[:24]), lambda: clef.rms_norm_quant(x[:, :144], w[:144], "fp8_h128"),
                 lambda: clef.rms_norm(x[:, 8:], w[8:].clone(), residual=None) and clef.rms_norm(x[:, 4:244], w[:240]),
                 lambda: clef.rms_norm(x[:1].expand(4, 256), w)):
        with pytest.raises(clef.ClefError) as e:
            call()
        assert e.value.status == 1


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("k", [528, 576, 1024, 5120, 5136, 8256, 16384, 16400, 17408, 17424, 32768])
def test_many_rows_have_the_bits_of_one(mode, k):
    """Calls whose CTAs keep rows ahead in shared memory, against calls of a row."""
    if mode.endswith("h128") and k % 128:
        k = k // 128 * 128
    m = 1300
    x, w, r = values((m, k), 30), weight(k, 31), values((m, k), 32)
    x[700] = (x[700].float() * 2.0 ** 70).to(torch.bfloat16)
    x[701] = 0
    r[701] = 0
    x[1299] = (x[1299].float() * 2.0 ** 100).to(torch.bfloat16)
    total, y = torch.empty_like(r), torch.empty_like(x)
    q, s = clef.rms_norm_quant(x, w, mode, residual=r, residual_out=total, y=y)
    assert torch.equal(total, (x.float() + r.float()).to(torch.bfloat16))
    assert torch.equal(clef.rms_norm(x, w, residual=r, residual_out=torch.empty_like(r)), y)
    for i in (0, 1, 151, 152, 455, 456, 700, 701, 702, 1298, 1299):
        yi = torch.empty_like(x[i:i + 1])
        qi, si = clef.rms_norm_quant(x[i:i + 1], w, mode, residual=r[i:i + 1].clone(), y=yi)
        assert torch.equal(qi[0], q[i]) and torch.equal(si[0], s[i]) and torch.equal(yi[0], y[i]), i
    keep = [i for i in range(0, m, 13) if i not in (700, 1299)]
    check_quant(q[keep], s[keep], mode, norm(x[keep], w, 1e-6, r[keep]), norm_rel(k))
    plain = clef.rms_norm_quant(x, w, mode)                                     # without a residual
    qi, si = clef.rms_norm_quant(x[9:10], w, mode)
    assert torch.equal(qi[0], plain[0][9]) and torch.equal(si[0], plain[1][9])
    assert clef.poll_status() == 0
