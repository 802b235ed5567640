"""Attention over pages whose value scales lie anywhere in fp32: values down to bf16's
smallest normal numbers, up to its largest, and both in one sequence.  Against fp64 with the
bounds of decode_util.attention."""
import numpy as np
import pytest
import torch

from decode_util import Cache, bf16, scattered_table
from test_gpu_kv_attention import check, run

pytestmark = pytest.mark.gpu

SIZES = {"tiny": (1e-37,), "tiny and normal": (1.0, 1e-37), "small and normal": (1.0, 1e-28), "large": (1e37,),
         "all": (1.0, 1e-37, 1e36, 1e-20, 1e18), "middle": (1e-12, 1e-25), "large and zero": (1e36, 0.0)}


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,n,len_,page", [(64, 1, 200, 16), (128, 1, 700, 32), (256, 1, 300, 16), (64, 10, 150, 16),
                                             (64, 40, 200, 16), (128, 150, 300, 64), (256, 40, 200, 32)])
@pytest.mark.parametrize("sizes", sorted(SIZES))
def test_value_scales(kind, dim, n, len_, page, sizes):
    """Pages of each size in turn, the softmax's weight spread over all of them or on those of one size."""
    rng = np.random.default_rng(dim + n + len_)
    table, pages = scattered_table(rng, [len_], page)
    size = np.asarray(SIZES[sizes])
    which = np.arange(len_) // page % len(size)
    for on in [None, *range(len(size))][:3]:
        c = Cache(kind, pages, 1, page, dim)
        new = rng.standard_normal((2, len_, 1, dim))
        new[0] *= np.where((on is None) | (which == on), 1.5, 0.01)[:, None, None]
        new[1] = np.clip(new[1], -3, 3) * size[which][:, None, None]
        new = bf16(new)
        c.append(table[0], len_, new)
        q = bf16(rng.standard_normal((n, 2, dim)) * 3)
        got, lse = run(rng, c, table, [len_], q)
        check(c, table, [len_], q, [0, n], got, lse)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("last", [1e-36, 1e36])
def test_one_page_at_the_end(kind, n, last):
    """The one page of another size comes after more pages than are looked up at a time, in
    sequences of one split and of many."""
    rng = np.random.default_rng(n)
    lens, page, dim = [1500, 9000, 33], 16, 64
    table, pages = scattered_table(rng, lens, page)
    c = Cache(kind, pages, 1, page, dim)
    for b, x in enumerate(lens):
        new = rng.standard_normal((2, x, 1, dim))
        new[1] *= np.where(np.arange(x) // page == (x - 1) // page - 1, last, 1.0)[:, None, None]
        c.append(table[b], x, bf16(np.clip(new, -3e38, 3e38)))
    q = bf16(rng.standard_normal((3 * n, 2, dim)))
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, np.arange(4) * n, got, lse)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("n,dim", [(1, 64), (1, 256), (5, 128), (33, 64), (200, 128), (33, 256)])
@pytest.mark.parametrize("amp,key", [(2.0 ** 110, 1e-33), (2.0 ** 116, 1e-35), (1e38, 1e-37), (1e-37, 1e36), (1e-20, 1e20)])
def test_query_and_key_sizes(kind, n, dim, amp, key):
    """Queries up to bf16's largest numbers over keys so small that the products are ordinary, and
    the other way round."""
    rng = np.random.default_rng(n + dim)
    lens, page = [140], 32
    table, pages = scattered_table(rng, lens, page)
    c = Cache(kind, pages, 1, page, dim)
    new = rng.standard_normal((2, 140, 1, dim))
    new[0] = np.clip(new[0], -3, 3) * key
    c.append(table[0], 140, bf16(new))
    q = bf16(np.clip(rng.standard_normal((n, 2, dim)), -3, 3) * amp)
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, [0, n], got, lse)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,len_", [(1, 40), (1, 1100), (5, 700), (40, 300), (20, 2300)])
@pytest.mark.parametrize("value", [0.5, 1e-30])
def test_queries_that_are_not_finite(kind, dim, n, len_, value):
    """An infinity or a NaN makes its own row and head NaN, and nothing else; rows that see nothing are zeros."""
    rng = np.random.default_rng(n + dim)
    lens, page = [len_, n - 1], 16
    table, pages = scattered_table(rng, lens, page)
    c = Cache(kind, pages, 1, page, dim)
    for b, x in enumerate(lens):
        new = rng.standard_normal((2, x, 1, dim))
        new[0] = -np.abs(new[0])                        # products with an infinity all of one sign
        new[1] *= value
        c.append(table[b], x, bf16(new))
    q = bf16(rng.standard_normal((2 * n, 2, dim)))
    ref, ref_lse = run(rng, c, table, lens, q)
    assert np.isfinite(ref).all()
    for bad in (np.inf, -np.inf, np.nan):
        p = q.copy()
        p[n // 2, 1, dim // 3] = bad
        p[n, 0, 0] = bad                                # the first row of the second sequence sees nothing
        got, lse = run(rng, c, table, lens, p)
        assert np.isnan(got[n // 2, 1]).all() and np.isnan(lse[n // 2, 1])
        assert not got[n, 0].any() and lse[n, 0] == -np.inf
        got[n // 2, 1], lse[n // 2, 1] = ref[n // 2, 1], ref_lse[n // 2, 1]
        assert np.array_equal(got, ref) and np.array_equal(lse, ref_lse)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("n", [1, 3, 24])
def test_many_items(kind, dim, n):
    """Several items a CTA, with and without pages of far sizes, some of them of zeros, in turn; each
    sequence as in a call of its own."""
    rng = np.random.default_rng(dim + n)
    lens = [int(x) for x in rng.integers(1, 170, 88)] + [1300, 700]
    page, heads = 16, 8
    table, pages = scattered_table(rng, lens, page)
    c = Cache(kind, pages, heads, page, dim)
    for b, x in enumerate(lens):
        new = rng.standard_normal((2, x, heads, dim))
        if b % 3:
            size = rng.choice([1.0, 1.0, 1e-37, 0.0, 1e36], (-(-x // page), heads))
            new[1] = np.clip(new[1], -3, 3) * size[np.arange(x) // page][..., None]
        c.append(table[b], x, bf16(new))
    q = bf16(rng.standard_normal((90 * n, 2 * heads, dim)))
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, np.arange(91) * n, got, lse)
    for b in (0, 1, 43, 88, 89):
        one, one_lse = run(rng, c, table[b:b + 1], lens[b:b + 1], q[b * n:(b + 1) * n])
        assert np.array_equal(one, got[b * n:(b + 1) * n]) and np.array_equal(one_lse, lse[b * n:(b + 1) * n])
