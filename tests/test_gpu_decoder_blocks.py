"""The decoder over block-scaled e4m3 weights, end to end: a layer's norms, linears, rotation, cache and attention run
together against 64 bits, and its steps, forks and captures."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from between_util import e4m3, f64, spread
from decode_util import Cache, attention, host_codes
from examples import decoder as module
from examples.decoder import Decoder

pytestmark = pytest.mark.gpu
HIDDEN, FF, HQ, HK, D, PAGE = 256, 384, 6, 2, 64, 16


def build(kind="int8", layers=2, seed=0, pages=40):
    g = torch.Generator().manual_seed(seed)

    def w(n, k):
        return (torch.randn(n, k, generator=g) * k ** -0.5).to(torch.bfloat16).cuda()

    def norm():
        return (1 + 0.2 * torch.randn(HIDDEN, generator=g)).to(torch.bfloat16).cuda()

    stack = [{"qkv": w((HQ + 2 * HK) * D, HIDDEN), "o": w(HIDDEN, HQ * D), "gateup": w(2 * FF, HIDDEN),
              "down": w(HIDDEN, FF), "norm_attn": norm(), "norm_mlp": norm()} for _ in range(layers)]
    return Decoder(stack, HQ, HK, D, sequences=6, pages=pages, width=12, page=PAGE, kind=kind, linears="fp8_block")


def rows(n, seed):
    return torch.randn(n, HIDDEN, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def values(pair, rows_of_scales):
    q, s = pair
    return e4m3(q) * spread(f64(s), rows_of_scales, q.shape)


def quantized(v):
    """What e4m3 codes in rows by 128 stand for."""
    t = torch.from_numpy(v).float()
    m, k = t.shape
    b = torch.nn.functional.pad(t, (0, -k % 128)).view(m, -1, 128)
    s = b.abs().amax(-1, keepdim=True) / 448
    q = (b / torch.where(s > 0, s, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).float() * s
    return q.view(m, -1)[:, :k].double().numpy()


def bf16(v):
    return torch.from_numpy(v).to(torch.bfloat16).double().numpy()


def layer(dec, i, x, at, cache, row, length):
    """One layer in 64 bits for the rows of one sequence, rounding where the library's tensors are of few bits."""
    w = {n: values(dec.fp8[i][n], 128) for n in module.NAMES}
    na, nm = (f64(t) for t in dec.norms[i])

    def normed(h, g):
        return quantized(h / np.sqrt((h * h).mean(-1, keepdims=True) + dec.eps) * g)

    qkv = bf16(normed(x, na) @ w["qkv"].T).reshape(-1, HQ + 2 * HK, D)
    t = at[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    a, b = qkv[:, : HQ + HK, : D // 2].copy(), qkv[:, : HQ + HK, D // 2:].copy()
    qkv[:, : HQ + HK] = bf16(np.concatenate((a * c - b * s, b * c + a * s), -1))
    cache.append(row, length, qkv[:, HQ:].reshape(-1, 2, HK, D).transpose(1, 0, 2, 3).astype(np.float32))
    o = bf16(attention(qkv[:, :HQ], cache.values(row, length), D ** -0.5, True)[0])
    mid = x + bf16(quantized(o.reshape(len(x), -1)) @ w["o"].T)
    gu = normed(mid, nm) @ w["gateup"].T
    h = bf16(gu[:, :FF] / (1 + np.exp(-gu[:, :FF])) * gu[:, FF:])
    return bf16(mid) + bf16(quantized(h) @ w["down"].T)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_a_layer_against_64_bits(kind):
    """A prompt and three answers' tokens of one sequence through one layer.  The model rounds where the library
    does, so that what differs are codes whose value lies within fp32 sums (or a bf16 step) of the border between
    two: each a code step on one of 256 or 384 products.  A code step of e4m3 is at most 1/8 of the value, a bf16 step of
    a code's input 2^-8 of it moves one code in 32 by a step; with normal values a product's sum so moves by
    (1 / 8) / sqrt(32) = 2.2% of its spread at most, three times in a row before the result, which adds as
    squares: 4%; the values of the result spread about 1."""
    dec = build(kind, layers=1)
    cache = Cache(kind, 40, HK, PAGE, D)
    got, want, length = [], [], 0
    for n, seed in ((37, 1), (1, 2), (1, 3), (1, 4)):
        x = rows(n, seed)
        got.append(f64(dec.prompt(x, {2: n}) if n > 1 else dec.step(x, [2])))
        assert clef.poll_status() == 0
        length += n
        want.append(layer(dec, 0, f64(x), np.arange(length - n, length, dtype=np.float64), cache, dec.table[2].tolist(), length))
    for a, b in zip(got, want):
        assert np.sqrt(((a - b) ** 2).mean()) <= 0.04 * np.sqrt((b ** 2).mean())
    # what has been cached are the layer's rotated keys: codes within a step of the model's
    k, _ = clef.kv_gather(dec.codes, dec.scales, dec.table, torch.full((length,), 2, dtype=torch.int32, device="cuda"),
                          torch.arange(length, dtype=torch.int32, device="cuda"))
    ref = cache.values(dec.table[2].tolist(), length)[0]
    assert np.sqrt(((f64(k) - ref) ** 2).mean()) <= 0.04 * np.sqrt((ref ** 2).mean())


def test_every_call_of_a_step(monkeypatch):
    """Two layers, three sequences: the calls of a step and their order."""
    dec = build()
    dec.prompt(rows(54, 1), {4: 37, 0: 1, 2: 16})
    calls = []
    names = ("rms_norm_quant", "fp8_block_linear", "rotary", "kv_append", "kv_attention", "quant_fp8_block", "fp8_block_gateup_swiglu")
    for name in names:
        inner = getattr(module, name)
        monkeypatch.setattr(module, name, lambda *a, inner=inner, name=name, **k: (calls.append(name), inner(*a, **k))[1])
    dec.step(rows(3, 2), [4, 0, 2])
    assert calls == 2 * ["rms_norm_quant", "fp8_block_linear", "rotary", "kv_append", "kv_attention", "quant_fp8_block",
                         "fp8_block_linear", "rms_norm_quant", "fp8_block_gateup_swiglu", "quant_fp8_block", "fp8_block_linear"]
    assert clef.poll_status() == 0


@pytest.mark.parametrize("length", [1, 16, 37])
def test_forked_answers(length):
    a, b = build(), build()
    p = rows(length, 7)
    out = a.prompt(p, {0: length})
    a.fork([0, 0], [2, 3])
    for s in (0, 2, 3):
        assert torch.equal(b.prompt(p, {s: length}), out)
    for t in range(20):
        x = rows(3, 10 + t)
        assert torch.equal(a.step(x, [0, 2, 3]), b.step(x, [0, 2, 3]))
    assert clef.poll_status() == 0 and a.lens.tolist() == [length + 20, 0, length + 20, length + 20, 0, 0]


def test_captured_step():
    a, b = build(), build()
    for d in (a, b):
        d.prompt(rows(30, 3), {0: 13, 1: 17})
    x = rows(2, 4)
    out = a.capture(x, [0, 1])
    for t in range(20):
        x.copy_(rows(2, 50 + t))
        a.replay()
        assert torch.equal(out, b.step(rows(2, 50 + t), [0, 1]))
    assert a.lens.tolist() == b.lens.tolist() and clef.poll_status() == 0


def test_input_is_left_alone():
    dec = build()
    x = rows(9, 5)
    was = x.clone()
    dec.prompt(x, {1: 9})
    assert torch.equal(x, was)
    with pytest.raises(ValueError):
        Decoder([], HQ, HK, D, 1, 1, 1, linears="fp8")
