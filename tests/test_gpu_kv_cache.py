"""Append and gather of the paged 8-bit cache: codes and scales equal, bit for
bit, to the rule in IEEE fp32, and every value within half a step of what was
written; the tokens of many calls, pages that end anywhere, zeros, extreme
magnitudes, strides, ragged rows, and indices out of range."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from decode_util import Cache, bf16, dev_bf16, dev_i32, host_codes, scattered_table

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3"]


def same(codes, scales, c):
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), c.scales.view(np.uint32))
    got = host_codes(codes)
    assert np.array_equal(got, c.codes), f"{(got != c.codes).sum()} codes differ"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 128), (2, 256)])
def test_many_calls(kind, page, heads, dim):
    """Sequences grown by calls of different sizes, the magnitudes rising and
    falling so that scales grow and stay."""
    rng = np.random.default_rng(page + heads + dim)
    ends = [[1, 2, 16, 17, 150], [0, 5, 5, 133, 134], [64, 64, 129, 200, 201]]
    table, pages = scattered_table(rng, [e[-1] for e in ends], page)
    c = Cache(kind, pages, heads, page, dim)
    codes, scales = c.device()
    tab, lens = dev_i32(table), [0, 0, 0]
    for call in range(5):
        now = [e[call] for e in ends]
        n = [a - b for a, b in zip(now, lens)]
        start = np.concatenate([[0], np.cumsum(n)])
        new = bf16(rng.standard_normal((2, start[-1], heads, dim)) * 10.0 ** rng.integers(-3, 3, (2, start[-1], heads, 1)))
        for b in range(3):
            if n[b]:
                c.append(table[b], now[b], new[:, start[b]:start[b + 1]])
        clef.kv_append(dev_bf16(new[0]), dev_bf16(new[1]), codes, scales, tab, dev_i32(now), dev_i32(start))
        same(codes, scales, c)
        lens = now
    assert clef.poll_status() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_values_are_near_what_was_written(kind):
    """In 64 bits: within half a step of the scale (int8), or half an e4m3 ulp
    (2^-4 of the value, 2^-10 steps below the normals), of a page written at once."""
    rng = np.random.default_rng(2)
    page, heads, dim, n = 32, 2, 128, 70
    table, pages = scattered_table(rng, [n], page)
    c = Cache(kind, pages, heads, page, dim)
    codes, scales = c.device()
    new = bf16(rng.standard_normal((2, n, heads, dim)))
    clef.kv_append(dev_bf16(new[0]), dev_bf16(new[1]), codes, scales, dev_i32(table), dev_i32([n]))
    k, v = clef.kv_gather(codes, scales, dev_i32(table), dev_i32([0] * n), dev_i32(np.arange(n)))
    s = scales.cpu().numpy().astype(np.float64)[:, table[0, np.arange(n) // page]][..., None]
    for pl, got in enumerate((k, v)):
        ref = new[pl].astype(np.float64)
        step = 0.5 * s[pl] if kind == "int8" else np.maximum(np.abs(ref) * 2.0 ** -4, s[pl] * 2.0 ** -10)
        tol = step * (1 + 2.0 ** -20) + np.abs(ref) * 2.0 ** -7     # and the bf16 of the output
        assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("kind", KINDS)
def test_zeros_and_extremes(kind):
    """All-zero pages (scale 0), then values; the smallest and largest magnitudes of bf16."""
    page, heads, dim = 16, 2, 64
    table = np.array([[2, 0]], np.int32)
    c = Cache(kind, 3, heads, page, dim)
    codes, scales = c.device()
    tab, at = dev_i32(table), 0
    steps = [np.zeros((2, 3, heads, dim)), np.full((2, 1, heads, dim), 1e-39), np.full((2, 2, heads, dim), -2e-38),
             np.full((2, 1, heads, dim), 3e38), np.zeros((2, 1, heads, dim)), np.full((2, 12, heads, dim), 1.0)]
    for new in steps:
        new = bf16(new)
        at += new.shape[1]
        c.append(table[0], at, new)
        clef.kv_append(dev_bf16(new[0]), dev_bf16(new[1]), codes, scales, tab, dev_i32([at]))
        same(codes, scales, c)
    assert clef.poll_status() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_strides_and_uniform_rows(kind):
    """Keys and values as column blocks of the packed projection's rows, and
    transposed to [heads][tokens]; the same number of rows for each sequence."""
    rng = np.random.default_rng(3)
    page, heads, dim, n = 64, 2, 128, 67
    lens = [70, 131, 67]
    table, pages = scattered_table(rng, lens, page)
    new = bf16(rng.standard_normal((2, 3 * n, heads, dim)))
    c = Cache(kind, pages, heads, page, dim, fill=0)
    c.scales[:] = 0.01
    codes, scales = c.device()
    more, sc = c.device()
    for b in range(3):
        c.append(table[b], lens[b], new[:, b * n:(b + 1) * n])
    wide = torch.zeros((3 * n, 5 * heads * dim), dtype=torch.bfloat16, device="cuda")
    k = wide[:, heads * dim:2 * heads * dim].view(3 * n, heads, dim)
    v = wide[:, 3 * heads * dim:4 * heads * dim].view(3 * n, heads, dim)
    k.copy_(dev_bf16(new[0]))
    v.copy_(dev_bf16(new[1]))
    clef.kv_append(k, v, codes, scales, dev_i32(table), dev_i32(lens))
    same(codes, scales, c)
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)
    vt = v.transpose(0, 1).contiguous().transpose(0, 1)
    clef.kv_append(kt, vt, more, sc, dev_i32(table), dev_i32(lens))
    same(more, sc, c)


def test_one_layer_of_a_pool():
    """Planes of a larger pool: the other layers keep their bytes."""
    rng = np.random.default_rng(4)
    pool = torch.randint(-127, 128, (3, 2, 5, 2, 16, 64), dtype=torch.int8, device="cuda")
    sc = torch.rand((3, 2, 5, 2), device="cuda")
    before, sb = pool.clone(), sc.clone()
    new = dev_bf16(rng.standard_normal((20, 2, 64)))
    clef.kv_append(new, new, pool[1], sc[1], dev_i32([[3, 1]]), dev_i32([20]))
    assert torch.equal(pool[0], before[0]) and torch.equal(pool[2], before[2])
    assert torch.equal(sc[0], sb[0]) and torch.equal(sc[2], sb[2])
    assert torch.equal(pool[1][:, [0, 2, 4]], before[1][:, [0, 2, 4]])
    k, v = clef.kv_gather(pool[1], sc[1], dev_i32([[3, 1]]), dev_i32([0] * 20), dev_i32(np.arange(20)))
    assert torch.equal(k, v) and (k - new).abs().max() < 0.05


def test_out_of_range_is_reported_and_left_out():
    codes = torch.zeros((2, 4, 1, 16, 64), dtype=torch.int8, device="cuda")
    scales = torch.zeros((2, 4, 1), device="cuda")
    new = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")

    def append(table, lens, start=None):
        codes.zero_(), scales.zero_()
        clef.kv_append(new, new, codes, scales, dev_i32(table), dev_i32(lens), None if start is None else dev_i32(start))
        return clef.poll_status(), sorted(set(torch.nonzero(scales[0, :, 0]).flatten().tolist()))

    assert append([[0], [3]], [1, 1]) == (0, [0, 3])
    assert append([[4], [3]], [1, 1]) == (5, [3])              # a page past the pool
    assert append([[-1], [3]], [1, 1]) == (5, [3])
    assert append([[0], [3]], [-2, 1]) == (5, [3])             # a negative length
    assert append([[0], [3]], [17, 1])[0] == 5                 # a length past the table's row
    assert append([[0], [3]], [0, 1]) == (5, [3])              # more rows than tokens
    assert append([[0], [3]], [1, 1], [0, 1, 3])[0] == 5       # rows past k
    assert append([[0], [3]], [1, 1], [0, -1, 2])[0] == 5
    assert append([[0], [3]], [1, 2], [0, 0, 2]) == (0, [3])   # a sequence without rows
    k, _ = clef.kv_gather(codes, scales, dev_i32([[0], [3]]), dev_i32([1, 2, -1, 1, 0]), dev_i32([0, 0, 0, 16, -1]))
    assert clef.poll_status() == 5
    assert k[0].any() and not k[1:].any()
    assert clef.poll_status() == 0


def test_refusals():
    codes = torch.zeros((2, 4, 2, 16, 64), dtype=torch.int8, device="cuda")
    scales = torch.zeros((2, 4, 2), device="cuda")
    new = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    ok = dict(k=new, v=new, codes=codes, scales=scales, table=dev_i32([[0], [1]]), lens=dev_i32([1, 1]))
    clef.kv_append(**ok)
    clef.kv_append(**{**ok, "k": new[:0], "v": new[:0]})
    for bad in (dict(k=new[:1]), dict(k=new.float()), dict(k=new[:, :1]), dict(codes=codes[:1]), dict(scales=scales[:, :3]),
                dict(codes=codes.transpose(2, 3)), dict(table=dev_i32([[0], [1]]).long()), dict(lens=dev_i32([1])),
                dict(row_start=dev_i32([0, 2])), dict(k=new[:1], v=new[:1]), dict(codes=codes.cpu()),
                dict(codes=codes.float())):
        with pytest.raises(ValueError):
            clef.kv_append(**{**ok, **bad})
    with pytest.raises(clef.ClefError):       # page of 24 tokens
        clef.kv_append(new, new, torch.zeros((2, 4, 2, 24, 64), dtype=torch.int8, device="cuda"), scales, ok["table"], ok["lens"])
    with pytest.raises(clef.ClefError):       # dim of 96
        clef.kv_append(torch.zeros((2, 2, 96), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 2, 96), dtype=torch.bfloat16, device="cuda"),
                       torch.zeros((2, 4, 2, 16, 96), dtype=torch.int8, device="cuda"), scales, ok["table"], ok["lens"])
    assert clef.poll_status() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("grows", ["now and then", "every token", "by half a step"])
def test_values_written_one_by_one(kind, page, grows):
    """The bound of include/clef.h with the scales that the page went through: half a step of each
    (int8), or 1/16 of the value as it was and 2^-10 of the scale each time (e4m3)."""
    rng = np.random.default_rng(page)
    heads, dim, n = 2, 64, page + 5
    table, pages = scattered_table(rng, [n], page)
    c = Cache(kind, pages, heads, page, dim)
    codes, scales = c.device()
    new = rng.standard_normal((2, n, heads, dim))
    if grows != "now and then":
        new *= (1.03 if grows == "every token" else 1 + 1 / 254) ** np.arange(n)[None, :, None, None]
    new = bf16(new)
    tab, seq = dev_i32(table), dev_i32([0] * n)
    history = np.zeros((n, 2, n, heads))                      # the scale of each token's page after each call
    at = table[0, np.arange(n) // page]
    for i in range(n):
        clef.kv_append(dev_bf16(new[0, i:i + 1]), dev_bf16(new[1, i:i + 1]), codes, scales, tab, dev_i32([i + 1]))
        history[i] = scales.cpu().numpy().astype(np.float64)[:, at]
    got = np.stack([t.double().cpu().numpy() for t in clef.kv_gather(codes, scales, tab, seq, dev_i32(np.arange(n)))])
    for t in range(n):
        s = history[t:, :, t]                                 # from the token's own append on
        fresh = np.concatenate([np.ones_like(s[:1], bool), np.diff(s, axis=0) > 0])
        total, g = (s * fresh).sum(0)[..., None], fresh.sum(0)[..., None] - 1
        v = np.abs(new[:, t].astype(np.float64))
        off = total / 2 if kind == "int8" else ((17 / 16) ** (g + 1) - 1) * v + total * (17 / 16) ** g * 2.0 ** -10
        off = off * (1 + 2.0 ** -16)                          # the fp32 roundings of scales, factors and products
        assert (np.abs(got[:, t] - new[:, t]) <= off + (v + off) * 2.0 ** -8).all(), t      # and the bf16 of the output
    assert clef.poll_status() == 0
