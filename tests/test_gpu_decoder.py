"""The decoder end to end: every 4-bit linear and attention call of its steps
against 64-bit models at their inputs, forks and moved pages leave the bits of
an answer alone, and a captured step replays as it ran.

Tolerances are those of the single operators: the 4-bit linear's (one bf16 ulp
and fp32 sums in 16-deep steps) and the attention's bound with one bf16 ulp; a
cached key or value is off by half a code step (int8) or 1/16 of itself (e4m3,
three bits; below its normal numbers half of 2^-9 of the scale), and by the
bf16 rounding of the gather."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from decode_util import Cache, attention, bf16_ulp, host_codes, w4_codes
from examples import decoder as module
from examples.decoder import Decoder

pytestmark = pytest.mark.gpu
HIDDEN, FF, HQ, HK, D, PAGE = 256, 384, 6, 2, 64, 16


def build(kind="int8", layers=2, group=64, seed=0, pages=40):
    g = torch.Generator().manual_seed(seed)

    def w(n, k):
        return (torch.randn(n, k, generator=g) * k ** -0.5).to(torch.bfloat16).cuda()

    stack = [{"qkv": w((HQ + 2 * HK) * D, HIDDEN), "o": w(HIDDEN, HQ * D), "gateup": w(2 * FF, HIDDEN),
              "down": w(HIDDEN, FF), "norm_attn": torch.ones(HIDDEN, dtype=torch.bfloat16).cuda(),
              "norm_mlp": torch.ones(HIDDEN, dtype=torch.bfloat16).cuda()} for _ in range(layers)]
    return Decoder(stack, HQ, HK, D, sequences=6, pages=pages, width=12, page=PAGE, kind=kind, group=group)


def rows(n, seed):
    return torch.randn(n, HIDDEN, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_steps_against_64_bits(kind, monkeypatch):
    dec = build(kind)
    dec.prompt(rows(54, 1), {4: 37, 0: 1, 2: 16})
    calls = []

    def recorded(name):
        inner = getattr(module, name)

        def call(*args):
            y = inner(*args)
            calls.append((name, [a.clone() if isinstance(a, torch.Tensor) else a for a in args], y))
            return y
        monkeypatch.setattr(module, name, call)

    for name in ("w4_linear", "kv_append", "kv_attention"):
        recorded(name)
    for t in range(3):
        dec.step(rows(3, 2 + t), [4, 0, 2])
    assert clef.poll_status() == 0
    assert dec.lens.tolist() == [4, 0, 19, 0, 40, 0]
    assert [c[0] for c in calls] == 6 * [
        "w4_linear", "kv_append", "kv_attention", "w4_linear", "w4_linear", "w4_linear"]
    for name, args, y in calls:
        if name == "w4_linear":
            x, qw, sw = args
            K, group = x.shape[1], x.shape[1] // sw.shape[1]
            w = w4_codes(qw.cpu().numpy(), K) * np.repeat(host(sw), group, 1)
            ref, mag = host(x) @ w.T, np.abs(host(x)) @ np.abs(w).T
            assert (np.abs(host(y) - ref) <= bf16_ulp(ref) + (K / 16 + 2) * 2.0 ** -23 * mag).all()
        elif name == "kv_append":
            k, v, codes, scales, table, lens, _ = args
            seq = torch.arange(3, dtype=torch.int32, device="cuda")
            got = clef.kv_gather(codes, scales, table, seq, lens - 1)
            step = host(torch.stack([scales[:, table[b, (int(lens[b]) - 1) // PAGE]] for b in range(3)], 1))[..., None]
            for new, at, s in zip((k, v), got, step):
                ref = host(new)
                off = 0.5 * s if kind == "int8" else np.maximum(np.abs(ref) / 16, 2.0 ** -10 * s)
                assert (np.abs(host(at) - ref) <= off * (1 + 2.0 ** -20) + bf16_ulp(ref)).all()
        else:
            q, codes, scales, table, lens, _ = args
            c = Cache(kind, codes.shape[1], HK, PAGE, D)
            c.codes, c.scales = host_codes(codes), scales.cpu().numpy()
            for b in range(3):
                kv = c.values(table[b].tolist(), int(lens[b]))
                ref, _, tol, _ = attention(host(q[b:b + 1]), kv, D ** -0.5, True)
                assert (np.abs(host(y[b:b + 1]) - ref) <= tol + bf16_ulp(ref)).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("length", [1, 16, 37])
def test_forked_answers(kind, length):
    """Three answers to one prompt, forked, with others freed and the pool
    compacted on the way, have the bits of three prompts read apart."""
    a, b = build(kind), build(kind)
    p = rows(length, 7)
    a.prompt(rows(20, 8), {5: 20})           # pages in front that go away
    out = a.prompt(p, {0: length})
    a.fork([0, 0], [2, 3])
    for s in (0, 2, 3):
        assert torch.equal(b.prompt(p, {s: length}), out)
    a.free([5])
    for t in range(20):
        if t == 9:
            live = a.compact()
            assert int(live) == int((a.refs > 0).sum()) and (a.refs[:int(live)] > 0).all()
        x = rows(3, 10 + t)
        if t < 3:
            x = x[:1].expand(3, -1).contiguous()       # the same token for each: the same bits
        ya, yb = a.step(x, [0, 2, 3]), b.step(x, [0, 2, 3])
        assert torch.equal(ya, yb)
        assert t >= 3 or (torch.equal(ya[0], ya[1]) and torch.equal(ya[0], ya[2]))
    assert clef.poll_status() == 0
    assert a.lens.tolist() == b.lens.tolist() == [length + 20, 0, length + 20, length + 20, 0, 0]
    a.free([0, 2, 3])
    assert not a.refs.any() and not a.lens.any()


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


def test_pool_too_small():
    """Recorded on the device; nothing is reserved."""
    dec = build(pages=2)
    dec.prompt(rows(32, 5), {0: 32})
    assert clef.poll_status() == 0
    clef.kv_reserve(dec.table, dec.lens, dec.refs, torch.ones_like(dec.lens), PAGE)
    assert clef.poll_status() == 6
    assert dec.lens.tolist() == [32, 0, 0, 0, 0, 0]


def test_refusals():
    dec = build()
    with pytest.raises(ValueError):
        dec.prompt(rows(3, 0), {0: 2})
    with pytest.raises(ValueError):
        dec.step(rows(2, 0), [0, 0])
    with pytest.raises(ValueError):
        dec.step(rows(2, 0), [0, 6])
    with pytest.raises(ValueError):
        dec.step(rows(1, 0), [0, 1])
    with pytest.raises(ValueError):
        Decoder([], HQ, HK, D, 1, 1, 1, kind="fp4")


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_a_full_pool_is_left_alone(kind, captured):
    """Two forks of a sequence whose last page is whole, and one free page: a step of both
    and a prompt that find no place leave every byte as it was; a step that has one is right."""
    a, b = build(kind, pages=3), build(kind)
    p = rows(32, 5)
    for d in (a, b):
        d.prompt(p, {0: 32})
    a.fork([0], [1])
    assert clef.poll_status() == 0
    x = rows(2, 6)
    if captured:
        a.capture(x, [0, 1])
    was = [t.clone() for t in (a.codes.view(torch.uint8), a.scales, a.table, a.lens, a.refs)]
    for call in range(3):
        if captured:
            a.replay()
        else:
            a.step(x, [0, 1])
        assert clef.poll_status() == 6
        assert all(torch.equal(t, w) for t, w in zip((a.codes.view(torch.uint8), a.scales, a.table, a.lens, a.refs), was))
    a.prompt(rows(40, 7), {1: 3, 2: 37})
    assert clef.poll_status() == 6
    assert all(torch.equal(t, w) for t, w in zip((a.codes.view(torch.uint8), a.scales, a.table, a.lens, a.refs), was))
    assert torch.equal(a.step(x[:1], [0]), b.step(x[:1], [0]))
    assert clef.poll_status() == 0 and a.lens.tolist() == [33, 32, 0, 0, 0, 0]
