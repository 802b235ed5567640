"""The cache where its numbers get large: code offsets past 32 bits, long
sequences of small pages, more items than CTAs in several rounds, lengths at
the edges of the splits.  Bounds are those of the operators' own tests."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from decode_util import dev_bf16, dev_i32, filled_cache, bf16
from test_gpu_kv_attention import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 30])
def test_offsets_past_32_bits(n):
    """The same sequences in a small pool and at the far end of one whose planes
    have 4.7 GB of codes each: the same bits from every call."""
    heads, page, dim, far = 8, 128, 128, 36000
    rng = np.random.default_rng(1)
    lens = [300 + n, 129 + n]
    kv = [dev_bf16(rng.standard_normal((sum(lens), heads, dim))) for _ in range(2)]
    new = [dev_bf16(rng.standard_normal((2 * n, heads, dim))) for _ in range(2)]
    q = dev_bf16(rng.standard_normal((2 * n, 2 * heads, dim)))
    got = []
    for pages, first in ((8, 0), (far, far - 8)):
        codes = torch.empty((2, pages, heads, page, dim), dtype=torch.int8, device="cuda")
        scales = torch.zeros((2, pages, heads), dtype=torch.float32, device="cuda")
        codes[:, first:] = 7
        table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4).flip(1).contiguous() + first
        start = dev_i32([0, lens[0], sum(lens)])
        clef.kv_append(*kv, codes, scales, table, dev_i32(lens), start)
        clef.kv_append(*new, codes, scales, table, dev_i32([x + n for x in lens]))
        last = dev_i32([x + n for x in lens])
        out = [clef.kv_attention(q, codes, scales, table, last)]
        seq = torch.arange(2, dtype=torch.int32, device="cuda")
        out += clef.kv_gather(codes, scales, table, seq, last - 1)
        spare = dev_i32([first + 4])                       # the second sequence has no fourth page
        clef.kv_copy_pages(codes, scales, table[0, :1].contiguous(), spare)
        out += [codes[:, first:].clone(), scales[:, first:].clone()]
        assert clef.poll_status() == 0
        assert torch.equal(codes[:, first + 4], codes[:, first + 3])
        got.append(out)
        del codes
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("n,len_,heads,group,page,dim", [
    (40, 4200, 1, 2, 16, 64), (33, 4097, 2, 1, 16, 128), (20, 3000, 1, 3, 16, 256), (130, 2050, 1, 1, 32, 256),
])
def test_long_many_rows(kind, n, len_, heads, group, page, dim):
    """Sequences cut in two or more, over page tables of several hundred entries;
    one just under the length that is cut."""
    rng = np.random.default_rng(len_ + dim)
    lens = [len_, 1920]
    c, table, _ = filled_cache(rng, kind, lens, heads, page, dim)
    q = bf16(rng.standard_normal((2 * n, heads * group, dim)) * 2)
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, [0, n, 2 * n], got, lse)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 24])
def test_many_items(n, dim):
    """Several items a CTA, some without a token, in a call of 90 sequences."""
    rng = np.random.default_rng(dim + n)
    lens = [int(x) for x in rng.integers(0, 150, 90)]
    lens[7] = 0
    c, table, _ = filled_cache(rng, "int8", lens, 8, 16, dim)
    q = bf16(rng.standard_normal((90 * n, 8, dim)))
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, np.arange(91) * n, got, lse)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 256])
def test_lengths_at_the_edges_of_splits(kind, dim):
    rng = np.random.default_rng(dim)
    lens = [511, 512, 513, 767, 768, 769, 1023, 1024, 1025, 1536, 1537]
    c, table, _ = filled_cache(rng, kind, lens, 1, 64, dim)
    q = bf16(rng.standard_normal((len(lens), 5, dim)))
    got, lse = run(rng, c, table, lens, q)
    check(c, table, lens, q, np.arange(len(lens) + 1), got, lse)


def test_first_call_of_a_shape_in_a_graph():
    """A 4-bit linear whose clusters are first sized while a stream is captured."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(13, 17408, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(96, 17408, generator=g) * 0.01).to(torch.bfloat16).cuda()
    qw, sw = clef.quant_w4(w, 64)
    y = torch.empty(13, 96, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clef.w4_linear(x, qw, sw, y=y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, clef.w4_linear(x, qw, sw)) and clef.poll_status() == 0
