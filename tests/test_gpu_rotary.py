"""Rotary positions against 64 bits, with angles from exact whole numbers."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from between_util import bf16_off, f64, rotary

pytestmark = pytest.mark.gpu


def heads(t, h, d, seed, spare=0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((t, (h + spare) * d), generator=g).to(torch.bfloat16).cuda()
    return wide[:, : h * d].view(t, h, d)


def positions(t, seed, far=2 ** 31 - 1):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, far, (t,), generator=g, dtype=torch.int64).to(torch.int32)
    p[0] = 0
    if t > 2:
        p[1], p[2] = 2 ** 31 - 1, -7
    return p.cuda()


def check(y, x, pos, turns, gain=1.0, interleaved=False):
    ref, off = rotary(x, pos.tolist(), turns.tolist(), gain, interleaved)
    assert (np.abs(f64(y) - ref) <= bf16_off(ref) + off).all()
    rot = 2 * turns.shape[0]
    assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,h,d,rot", [(1, 1, 8, 2), (3, 56, 128, 128), (1, 8, 64, 64), (7, 5, 80, 32), (65, 3, 96, 96), (5, 2, 256, 64),
                                       (9, 4, 128, 122), (4, 1, 64, 24), (3, 7, 72, 72), (2, 1024, 16, 16), (300, 2, 1024, 512),
                                       (700, 12, 128, 128)])
def test_rotary(t, h, d, rot, interleaved):
    x, pos = heads(t, h, d, 1, spare=2), positions(t, 2)
    turns = clef.rotary_turns(rot, 500000.0)
    for gain in (1.0, 1.37):
        check(clef.rotary(x, pos, turns, gain, interleaved), x, pos, turns, gain, interleaved)
    own = x.clone(memory_format=torch.contiguous_format)
    assert clef.rotary(own, pos, turns, interleaved=interleaved, out=own) is own       # in place
    assert torch.equal(own, clef.rotary(x, pos, turns, interleaved=interleaved))
    assert clef.poll_status() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_leaves_the_rest_of_a_row(interleaved):
    wide = torch.randn((11, 6, 128), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    was, pos, turns = wide.clone(), positions(11, 4, 5000), clef.rotary_turns(64)
    clef.rotary(wide[:, 1:5], pos, turns, interleaved=interleaved, out=wide[:, 1:5])
    assert torch.equal(wide[:, :1], was[:, :1]) and torch.equal(wide[:, 5:], was[:, 5:])
    check(wide[:, 1:5], was[:, 1:5], pos, turns, 1.0, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 48, 50])
def test_orders_of_tokens_and_heads(interleaved, rot):
    """Heads of tokens, tokens of heads, on either side."""
    x, pos, turns = heads(37, 4, 64, 5), positions(37, 6), clef.rotary_turns(rot, 10000.0)
    want = clef.rotary(x, pos, turns, 1.0, interleaved)
    other = x.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    out = torch.empty((4, 37, 64), dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)
    assert torch.equal(clef.rotary(other, pos, turns, 1.0, interleaved, out=out), want) and torch.equal(out, want)


def test_turned_back():
    """Negative positions turn back: twice rounded, the values again."""
    x, pos, turns = heads(50, 3, 128, 7), positions(50, 8, 100000), clef.rotary_turns(128)
    back = clef.rotary(clef.rotary(x, pos, turns), -pos, turns)
    a, b = f64(x)[..., :64], f64(x)[..., 64:]
    # the first rounding turns with its pair: half a bf16 step of either; then its own
    size = np.sqrt(a * a + b * b) * np.sqrt(2.0) * 2.0 ** -8 * 2
    assert (np.abs(f64(back) - f64(x)) <= np.concatenate([size, size], -1) * 1.01 + 2.0 ** -20).all()


def test_far_offsets():
    """Tokens whose values lie past 2^32 bytes."""
    t, h, d = 5, 2, 128
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("memory")
    pitch = 2 ** 29 + 8
    big = torch.empty(4 * pitch + h * d, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((t, h, d), (pitch, d, 1))
    x.copy_(heads(t, h, d, 9))
    pos, turns = positions(t, 10), clef.rotary_turns(d)
    assert torch.equal(clef.rotary(x, pos, turns), clef.rotary(x.contiguous(), pos, turns))


def test_scaled_tables_rotate():
    x, pos = heads(40, 2, 128, 11), positions(40, 12, 10 ** 6)
    for scaling in ("linear", "theta", "by_parts"):
        turns = clef.rotary_turns(128, 10000.0, scaling, 16.0)
        check(clef.rotary(x, pos, turns), x, pos, turns)


def test_empty_stream_and_graph():
    turns = clef.rotary_turns(64)
    e = torch.empty((0, 3, 64), dtype=torch.bfloat16, device="cuda")
    assert clef.rotary(e, torch.empty(0, dtype=torch.int32, device="cuda"), turns).shape == (0, 3, 64)
    x, pos = heads(6, 4, 64, 13), positions(6, 14)
    want = clef.rotary(x, pos, turns)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = clef.rotary(x, pos, turns, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = clef.rotary(x, pos, turns)
    for seed in (15, 16):
        pos.copy_(positions(6, seed))
        graph.replay()
        assert torch.equal(got, clef.rotary(x, pos, turns))


def test_refusals():
    x, pos, turns = heads(4, 2, 64, 17), positions(4, 18), clef.rotary_turns(64)
    for call in (lambda: clef.rotary(x, pos.long(), turns), lambda: clef.rotary(x, pos[:3], turns),
                 lambda: clef.rotary(x, pos, turns.int()), lambda: clef.rotary(x, pos, clef.rotary_turns(66)),
                 lambda: clef.rotary(x, pos, turns[:0]), lambda: clef.rotary(x.float(), pos, turns),
                 lambda: clef.rotary(x[0], pos, turns), lambda: clef.rotary(x, pos, turns, out=x[:3]),
                 lambda: clef.rotary(x, pos, turns.cpu()),
                 lambda: clef.rotary(x, pos, turns, out=torch.empty_like(x).as_strided((4, 2, 64), (64, 64, 1)))):
        with pytest.raises(ValueError):
            call()
    off = x.contiguous().view(-1)[4:].as_strided((3, 2, 56), (128, 64, 1))       # 8-byte aligned
    for call in (lambda: clef.rotary(x, pos, turns, float("inf")), lambda: clef.rotary(x[..., :60], pos, turns[:8]),
                 lambda: clef.rotary(x[:, :1].expand(4, 2, 64), pos, turns),
                 lambda: clef.rotary(x, pos, turns, out=x[:, :1].expand(4, 2, 64)), lambda: clef.rotary(off, pos[:3], turns[:16])):
        with pytest.raises(clef.ClefError) as e:
            call()
        assert e.value.status == 1
