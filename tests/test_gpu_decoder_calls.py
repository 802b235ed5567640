"""Every call that the decoder over block-scaled e4m3 weights makes, on the inputs that it makes it with, against 64 bits:
norms, linears, rotation, cache, attention and quantizers of a prompt and of single tokens, each within its own roundings."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from between_util import block_amax, check_codes, e4m3, f64, norm, norm_rel, spread
from decode_util import Cache, attention, bf16_ulp, host_codes
from examples import decoder as module
from test_gpu_decoder_blocks import D, HK, PAGE, build, rows
from test_gpu_fp8_block import check_gateup, check_linear
from test_gpu_norm import check_quant
from test_gpu_rotary import check as check_rotary

pytestmark = pytest.mark.gpu


def pool(codes, scales, kind):
    c = Cache(kind, codes.shape[1], HK, PAGE, D)
    c.codes, c.scales = host_codes(codes), scales.cpu().numpy().copy()
    return c


def check_norm_call(inner, x, w, mode, eps, residual=None):
    before = None if residual is None else residual.clone()
    q, s = inner(x, w, mode, eps, **({} if residual is None else {"residual": residual}))
    check_quant(q, s, mode, norm(x, w, eps, before), norm_rel(x.shape[1]))
    assert residual is None or torch.equal(residual, (x.float() + before.float()).to(torch.bfloat16))
    return q, s


def check_linear_call(inner, qx, sx, qw, sw):
    y = inner(qx, sx, qw, sw)
    check_linear(y, (qx, sx, qw, sw, None))
    return y


def check_gateup_call(inner, qx, sx, qw, sw):
    h = inner(qx, sx, qw, sw)
    check_gateup(h, (qx, sx, qw, sw, None))
    return h


def check_quant_call(inner, x):
    q, s = inner(x)
    v = f64(x)
    amax = spread(block_amax(v, 1), 1, v.shape)
    check_codes(e4m3(q), spread(f64(s), 1, v.shape), v, amax, 448.0, np.zeros_like(v))
    return q, s


def check_rotary_call(inner, x, at, turns, out):
    assert out is x
    before = x.clone()
    inner(x, at, turns, out=out)
    check_rotary(x, before, at, turns)
    return x


def spans(table, lens, start, rows):
    """(sequence, its first row, rows, page row, length) of a call."""
    start = list(range(len(lens) + 1)) if start is None else start.tolist()
    return [(b, start[b], start[b + 1] - start[b], table[b].tolist(), int(lens[b])) for b in range(len(lens))]


def append_call(kind):
    def call(inner, k, v, codes, scales, table, lens, placed):
        c = pool(codes, scales, kind)
        inner(k, v, codes, scales, table, lens, placed)
        new = np.stack([f64(k), f64(v)]).astype(np.float32)
        for _, first, n, row, length in spans(table, lens, placed, len(k)):
            if n:
                c.append(row, length, new[:, first:first + n])
        assert np.array_equal(host_codes(codes), c.codes) and np.array_equal(scales.cpu().numpy(), c.scales)
    return call


def attention_call(kind):
    def call(inner, q, codes, scales, table, lens, start):
        o = inner(q, codes, scales, table, lens, start)
        c, q64, got = pool(codes, scales, kind), f64(q), f64(o)
        for _, first, n, row, length in spans(table, lens, start, len(q)):
            ref, _, tol, _ = attention(q64[first:first + n], c.values(row, length), D ** -0.5, True)
            assert (np.abs(got[first:first + n] - ref) <= tol + bf16_ulp(ref)).all()
        return o
    return call


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_each_call_on_its_own_inputs(kind, monkeypatch):
    dec = build(kind)
    calls = []
    checks = {"rms_norm_quant": check_norm_call, "fp8_block_linear": check_linear_call, "fp8_block_gateup_swiglu": check_gateup_call,
              "quant_fp8_block": check_quant_call, "rotary": check_rotary_call, "kv_append": append_call(kind),
              "kv_attention": attention_call(kind)}
    for name, check in checks.items():
        inner = getattr(module, name)
        monkeypatch.setattr(module, name, lambda *a, inner=inner, check=check, name=name, **k: (calls.append(name), check(inner, *a, **k))[1])
    dec.prompt(rows(54, 1), {4: 37, 0: 1, 2: 16})
    for t in range(3):
        dec.step(rows(3, 2 + t), [4, 0, 2])
    dec.prompt(rows(9, 8), {2: 9})
    assert len(calls) == 5 * 22 and set(calls) == set(checks) and clef.poll_status() == 0
