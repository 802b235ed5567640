"""The places of partial results when the sequences of a call have any number of rows: nothing is
written outside of them, and every sequence has the bits of a call of its own."""
import ctypes as C

import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from decode_util import dev_bf16, dev_i32, filled_cache

pytestmark = pytest.mark.gpu


def attend(q, codes, scales, table, lens, start, out, lse, slack=1 << 20):
    """clef_kv_attention with a workspace of the size asked for and a border behind it."""
    L, need = clef.library(), C.c_int64(-1)
    rows, hq, d = q.shape
    _, pages, h, page, _ = codes.shape
    seqs, width = table.shape
    assert L.clef_kv_attention_workspace(rows, 1, seqs, hq, h, d, width * page, C.byref(need)) == 0
    ws = torch.full((need.value + slack,), 0xA5, dtype=torch.uint8, device="cuda")

    def p(t):
        return C.c_void_p(t.data_ptr())
    rc = L.clef_kv_attention(p(q), hq * d, d, rows, p(start), hq, 0, p(codes), codes.stride(0), p(scales), scales.stride(0),
                             pages, h, page, d, p(table), width, seqs, width, p(lens), d ** -0.5, 1, p(out), hq * d, d, p(lse),
                             p(ws), need, C.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0 and clef.poll_status() == 0
    assert (ws[need.value:] == 0xA5).all()


@pytest.mark.parametrize("heads,group,dim", [(2, 4, 64), (1, 8, 128), (4, 1, 256)])
@pytest.mark.parametrize("n", [
    [1, 1, 1, 1, 1, 1], [1, 1, 70, 1, 1, 1], [40, 0, 1, 40, 3, 17], [0, 0, 0, 0, 0, 90], [300, 1, 5, 0, 1, 200],
])
def test_rows_of_any_number(heads, group, dim, n):
    rng = np.random.default_rng(dim + sum(n))
    lens = [9000, 600, 2600, 1025, 300, 4200]
    c, table, _ = filled_cache(rng, "int8", lens, heads, 64, dim)
    codes, scales = c.device()
    tab, ln = dev_i32(table), dev_i32(lens)
    start = np.concatenate([[0], np.cumsum(n)])
    hq = heads * group
    q = dev_bf16(rng.standard_normal((sum(n), hq, dim)))
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    attend(q, codes, scales, tab, ln, dev_i32(start), out, lse)
    assert torch.equal(out, clef.kv_attention(q, codes, scales, tab, ln, dev_i32(start)))
    for b in range(6):
        r = slice(int(start[b]), int(start[b + 1]))
        if n[b]:
            one_lse = torch.zeros((n[b], hq), device="cuda")
            one = clef.kv_attention(q[r], codes, scales, tab[b:b + 1], ln[b:b + 1], lse=one_lse)
            assert torch.equal(out[r], one) and torch.equal(lse[r], one_lse)
    assert clef.poll_status() == 0
