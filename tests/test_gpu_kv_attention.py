"""Attention over the paged 8-bit cache against fp64 on the values the codes
stand for; the tolerance is decode_util.attention's bound plus one bf16 ulp."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from decode_util import Cache, attention, bf16, bf16_ulp, dev_bf16, dev_i32, filled_cache, scattered_table

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3"]


def run(rng, c, table, lens, q, start=None, causal=True, scale=None, **kw):
    codes, scales = c.device()
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = clef.kv_attention(dev_bf16(q), codes, scales, dev_i32(table), dev_i32(lens),
                            None if start is None else dev_i32(start), scale, causal, lse=lse, **kw)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def check(c, table, lens, q, start, got, lse, causal=True, scale=None):
    scale = c.D ** -0.5 if scale is None else scale
    for b, x in enumerate(lens):
        r = slice(start[b], start[b + 1])
        o, ls, tol, tl = attention(q[r].astype(np.float64), c.values(table[b], x), scale, causal)
        bad = ~(np.abs(got[r] - o) <= tol + bf16_ulp(o))
        assert not bad.any(), (b, x, int(bad.sum()), float((np.abs(got[r] - o) / (tol + bf16_ulp(o))).max()))
        none = np.isinf(ls)
        assert np.array_equal(none, np.isinf(lse[r])) and (lse[r][none] < 0).all() and not got[r][none].any()
        assert (np.abs(lse[r][~none] - ls[~none]) <= tl[~none]).all()
    assert clef.poll_status() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,group", [(2, 1), (1, 6), (2, 8), (1, 16)])
def test_single_tokens(kind, dim, page, heads, group):
    """One query a sequence, lengths from none to past a split."""
    rng = np.random.default_rng(dim + page + group)
    lens = [0, 1, 15, 16, 17, 128, 129, 300, 517]
    c, table, _ = filled_cache(rng, kind, lens, heads, page, dim)
    q = bf16(rng.standard_normal((len(lens), heads * group, dim)))
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, np.arange(len(lens) + 1), got, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,group,page", [(2, 3, 16), (1, 8, 64), (1, 1, 128)])
def test_ragged_queries(kind, dim, causal, heads, group, page):
    """No, one, a few and many queries a sequence in one call; more queries than
    tokens (whose first rows see nothing); an empty sequence."""
    rng = np.random.default_rng(dim + group)
    lens, n = [5, 40, 300, 131, 0, 260, 3, 64], [5, 1, 0, 17, 2, 150, 6, 2]
    start = np.concatenate([[0], np.cumsum(n)])
    c, table, _ = filled_cache(rng, kind, lens, heads, page, dim)
    q = bf16(rng.standard_normal((start[-1], heads * group, dim)) * 2)
    got, lse = run(rng, c, table, lens, q, start, causal)
    check(c, table, lens, q, start, got, lse, causal)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("len_,dim", [(2048, 64), (2049, 128), (8200, 64), (33000, 64)])
def test_long(kind, len_, dim):
    """Each length of a split, and the join of many."""
    rng = np.random.default_rng(len_)
    lens = [len_, 100]
    c, table, _ = filled_cache(rng, kind, lens, 1, 128, dim)
    q = bf16(rng.standard_normal((2, 4, dim)))
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, np.arange(3), got, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,len_,heads,group,page", [
    (17, 17, 1, 1, 16), (128, 128, 2, 1, 32), (129, 200, 1, 1, 64), (257, 300, 1, 1, 128), (100, 700, 2, 5, 16),
    (33, 1025, 1, 4, 64), (20, 2500, 2, 1, 128), (300, 1100, 1, 2, 32),
])
def test_many_rows(kind, dim, n, len_, heads, group, page):
    """One and two row tiles, partly filled ones, one and more steps, sequences
    cut along their tokens and joined; a second sequence beside the first."""
    rng = np.random.default_rng(n + len_ + dim)
    lens = [len_, max(n, len_ // 3)]
    c, table, _ = filled_cache(rng, kind, lens, heads, page, dim)
    q = bf16(rng.standard_normal((2 * n, heads * group, dim)) * 2)
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, [0, n, 2 * n], got, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 40])
def test_scales_far_apart(kind, n):
    """Value scales 10^12 apart in one sequence, the weight on the small pages
    or on the large ones; key scales apart too; a page of zeros."""
    rng = np.random.default_rng(11)
    page, dim, L = 16, 64, 160
    table, pages = scattered_table(rng, [L], page)
    for big in (0, 5, 9):
        c = Cache(kind, pages, 1, page, dim)
        new = bf16(rng.standard_normal((2, L, 1, dim)))
        at = np.arange(L) // page
        new[1] *= np.where(at == big, 1e6, 1e-6)[:, None, None].astype(np.float32)
        new[1][at == 3] = 0
        new[0] *= np.where(at == big, 0.01, 3.0)[:, None, None].astype(np.float32)
        new = bf16(new)
        c.append(table[0], L, new)
        q = bf16(rng.standard_normal((n, 2, dim)) * 4)
        got, lse = run(rng, c, table, [L], q, causal=False)
        check(c, table, [L], q, [0, n], got, lse, causal=False)


@pytest.mark.parametrize("n", [1, 33])
@pytest.mark.parametrize("amp", [1e-30, 1.0, 50.0, 3e4])
def test_query_magnitudes(n, amp):
    """Queries from tiny to such that one token takes all the weight."""
    rng = np.random.default_rng(12)
    lens = [70]
    c, table, _ = filled_cache(rng, "int8", lens, 2, 32, 128)
    q = bf16(rng.standard_normal((n, 4, 128)) * amp)
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, [0, n], got, lse)


@pytest.mark.parametrize("n", [1, 24])
def test_scale_argument(n):
    rng = np.random.default_rng(13)
    lens = [90, 31]
    c, table, _ = filled_cache(rng, "e4m3", lens, 1, 16, 64)
    q = bf16(rng.standard_normal((2 * n, 2, 64)))
    for scale in (0.0, 1.0, -0.5):
        got, lse = run(rng, c, table, lens, q, scale=scale)
        check(c, table, lens, q, [0, n, 2 * n], got, lse, scale=scale)


@pytest.mark.parametrize("n", [1, 5, 200])
def test_strides_streams_and_repeats(n):
    """Queries as a column block of the packed projection's rows, outputs into a
    wider buffer and as [heads][tokens], a side stream; the same bits each time."""
    rng = np.random.default_rng(14)
    lens, heads, group, dim = [333, 210], 2, 3, 128
    c, table, _ = filled_cache(rng, "int8", lens, heads, 64, dim)
    codes, scales = c.device()
    tab, ln = dev_i32(table), dev_i32(lens)
    hq = heads * group
    q = dev_bf16(rng.standard_normal((2 * n, hq, dim)))
    ref = clef.kv_attention(q, codes, scales, tab, ln)
    wide = torch.zeros((2 * n, (hq + 4) * dim), dtype=torch.bfloat16, device="cuda")
    wide[:, : hq * dim] = q.view(2 * n, -1)
    out = torch.zeros((2 * n, hq + 1, dim), dtype=torch.bfloat16, device="cuda")
    assert clef.kv_attention(wide[:, : hq * dim].view(2 * n, hq, dim), codes, scales, tab, ln, out=out[:, :hq]) is not None
    assert torch.equal(out[:, :hq], ref) and not out[:, hq].any()
    ht = torch.zeros((hq, 2 * n, dim), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    clef.kv_attention(q, codes, scales, tab, ln, out=ht)
    assert torch.equal(ht, ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [clef.kv_attention(q, codes, scales, tab, ln, stream=side) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(o, ref) for o in got)


@pytest.mark.parametrize("n", [1, 3, 40])
def test_a_sequence_does_not_depend_on_the_others(n):
    rng = np.random.default_rng(15)
    lens = [260, 64, 700, 40]
    c, table, _ = filled_cache(rng, "e4m3", lens, 2, 32, 128)
    codes, scales = c.device()
    q = dev_bf16(rng.standard_normal((4 * n, 8, 128)))
    start = dev_i32(np.arange(5) * n)
    whole = clef.kv_attention(q, codes, scales, dev_i32(table), dev_i32(lens))
    assert torch.equal(whole, clef.kv_attention(q, codes, scales, dev_i32(table), dev_i32(lens), start))
    for b in range(4):
        one = clef.kv_attention(q[b * n:(b + 1) * n], codes, scales, dev_i32(table[b:b + 1]), dev_i32(lens[b:b + 1]))
        assert torch.equal(one, whole[b * n:(b + 1) * n])


def test_graph():
    """Captured once, replayed as the lengths grow: nothing about them is kept on the host."""
    rng = np.random.default_rng(16)
    c, table, _ = filled_cache(rng, "int8", [500], 2, 64, 128)
    codes, scales = c.device()
    q = dev_bf16(rng.standard_normal((1, 12, 128)))
    tab, ln = dev_i32(table), dev_i32([3])
    out = clef.kv_attention(q, codes, scales, tab, ln)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clef.kv_attention(q, codes, scales, tab, ln, out=out)
    for x in (1, 128, 129, 500):
        ln.fill_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, clef.kv_attention(q, codes, scales, tab, dev_i32([x])))


@pytest.mark.parametrize("n", [1, 30])
def test_out_of_range_is_reported(n):
    """Pages and lengths out of range fault nothing; the other sequences are right."""
    rng = np.random.default_rng(17)
    lens = [100, 90]
    c, table, pages = filled_cache(rng, "int8", lens, 1, 16, 64)
    codes, scales = c.device()
    q = dev_bf16(rng.standard_normal((2 * n, 2, 64)))
    ref = clef.kv_attention(q, codes, scales, dev_i32(table), dev_i32(lens))
    for edit in (lambda t, x: t.__setitem__((0, 2), pages), lambda t, x: t.__setitem__((0, 0), -5),
                 lambda t, x: x.__setitem__(0, -1), lambda t, x: x.__setitem__(0, 10 ** 9)):
        t, x = table.copy(), list(lens)
        edit(t, x)
        out = clef.kv_attention(q, codes, scales, dev_i32(t), dev_i32(x))
        assert clef.poll_status() == 5
        assert torch.equal(out[n:], ref[n:])
    for start in ([0, n, 2 * n + 1], [-1, n, 2 * n], [n, 0, 2 * n]):
        clef.kv_attention(q, codes, scales, dev_i32(table), dev_i32(lens), dev_i32(start))
        assert clef.poll_status() == 5
    assert clef.poll_status() == 0


def test_waits_run_out():
    """The test knob makes the tile kernel's products wait for what never comes:
    the waits give up, the status says so, and the next call is right."""
    rng = np.random.default_rng(18)
    c, table, _ = filled_cache(rng, "int8", [300], 2, 64, 128)
    codes, scales = c.device()
    q = dev_bf16(rng.standard_normal((50, 4, 128)))
    args = (q, codes, scales, dev_i32(table), dev_i32([300]))
    ref = clef.kv_attention(*args)
    clef.set_wait_limit_ns(2_000_000)
    clef.test_force_timeout(True)
    try:
        clef.kv_attention(*args)
        assert clef.poll_status() == 4
    finally:
        clef.test_force_timeout(False)
        clef.set_wait_limit_ns(1_000_000_000)
    assert torch.equal(clef.kv_attention(*args), ref) and clef.poll_status() == 0


def test_refusals():
    codes = torch.zeros((2, 4, 2, 16, 64), dtype=torch.int8, device="cuda")
    scales = torch.zeros((2, 4, 2), device="cuda")
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    ok = dict(q=q, codes=codes, scales=scales, table=dev_i32([[0], [1]]), lens=dev_i32([1, 1]))
    clef.kv_attention(**ok)
    assert clef.kv_attention(**{**ok, "q": q[:0]}).shape == (0, 4, 64)
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[:, :, :32]), dict(q=q[:1]), dict(codes=codes[:1]),
                dict(out=q[:1]), dict(out=q.float()), dict(lse=torch.zeros((2, 3), device="cuda")),
                dict(lens=dev_i32([1])), dict(row_start=dev_i32([0, 2])),
                dict(out=torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda").expand(2, 4, 64))):
        with pytest.raises(ValueError):
            clef.kv_attention(**{**ok, **bad})
    for scale in (float("nan"), float("inf")):
        with pytest.raises(clef.ClefError):
            clef.kv_attention(**ok, scale=scale)
    assert clef.poll_status() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("mean", [0.0, 3.0])
def test_one_large_key_a_page_and_queries_with_a_mean(kind, dim, n, mean):
    """The page's key scale is set by one token, the other codes are a few steps: the sums of
    int8 keys of few rows run over c + 128, whose fp32 rounding goes by 128 scale sum |q| beside
    that of the products."""
    rng = np.random.default_rng(dim + n)
    lens, page = [150], 16
    table, pages = scattered_table(rng, lens, page)
    c = Cache(kind, pages, 1, page, dim)
    new = rng.standard_normal((2, 150, 1, dim))
    new[0, 3::page] *= 40
    c.append(table[0], 150, bf16(new))
    q = bf16(rng.standard_normal((n, 2, dim)) + mean)
    got, lse = run(rng, c, table, lens, q)
    kv = c.values(table[0], 150)
    ref, ls, tol, tl = attention(q.astype(np.float64), kv, dim ** -0.5, True)
    most = c.scales[0, table[0, :-(-150 // page)]].max()
    dx = dim ** -0.5 * (dim / 16 + 4) * 2.0 ** -23 * 128 * most * np.abs(q).sum(-1, dtype=np.float64)
    worst = np.abs(kv[1]).max(0)[0]
    tol = tol + np.expm1(2 * dx)[..., None] * worst
    assert (np.abs(got - ref) <= tol + bf16_ulp(ref)).all()
    assert (np.abs(lse - ls) <= tl + dx).all()
    assert clef.poll_status() == 0
