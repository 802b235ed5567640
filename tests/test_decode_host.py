"""Host-side refusals of the token-by-token operators, without a GPU: the C ABI
answers bad arguments before it touches a device, empty calls return CLEF_OK,
and the workspace sizes follow the shapes."""
import ctypes as C

import numpy as np
import pytest

import w8a8_quantized_projections_gb300 as clef
from decode_util import w4_codes, w4_pack

P = C.c_void_p(0x10000)          # 16-byte aligned, never dereferenced
ODD = C.c_void_p(0x10002)
NUL = C.c_void_p(None)
FAR = 1 << 40


def edits(good, bad):
    for at, value in bad:
        args = list(good)
        args[at] = value
        yield at, value, args


def refused(fn, good, bad):
    for at, value, args in edits(good, bad):
        assert fn(*args) == 1, (at, value)


def test_w4():
    L = clef.library()
    quant = [P, 64, 256, 256, 64, P, P, NUL]
    refused(L.clef_quant_w4, quant, [(0, NUL), (0, ODD), (1, -1), (1, FAR), (2, 0), (2, 252), (3, 248), (3, 260),
                                     (4, 16), (5, NUL), (5, ODD), (6, NUL), (6, ODD)])
    assert L.clef_quant_w4(NUL, 0, 256, 256, 64, NUL, NUL, NUL) == 0
    lin = [P, 256, P, P, 128, NUL, 4, 64, 256, P, 64, NUL]
    refused(L.clef_w4_linear, lin, [(0, NUL), (0, ODD), (1, 248), (1, 260), (2, NUL), (2, ODD), (3, ODD), (4, 0), (4, 256),
                                    (5, C.c_void_p(0x10001)), (6, -1), (6, FAR), (7, 0), (7, FAR), (8, 0), (8, 12), (8, 65544),
                                    (9, NUL), (9, C.c_void_p(0x10001)), (10, 63)])
    assert L.clef_w4_linear(NUL, 256, P, P, 128, NUL, 0, 64, 256, NUL, 64, NUL) == 0


#       codes plane scales plane pages heads page dim
LAYER = [P, 4 * 2 * 16 * 64, P, 4 * 2, 4, 2, 16, 64]
LAYER_BAD = [(0, NUL), (0, ODD), (1, 4 * 2 * 16 * 64 - 16), (1, 4 * 2 * 16 * 64 + 8), (2, NUL), (2, ODD), (3, 7), (4, -1),
             (4, FAR), (5, 0), (5, 1025), (6, 8), (6, 48), (6, 256), (7, 32), (7, 96), (7, 512)]
#       table ldt seqs width
TABLE = [P, 3, 2, 3]
TABLE_BAD = [(0, NUL), (0, ODD), (1, 2), (2, -1), (2, 4097), (3, -1), (3, 1 << 21)]


def at(offset, bad):
    return [(offset + i, v) for i, v in bad]


def test_append_and_gather():
    L = clef.library()
    app = [P, 128, 64, P, 128, 64, 4, NUL, 0, *LAYER, *TABLE, P, NUL]
    refused(L.clef_kv_append, app, [(0, NUL), (0, ODD), (1, 130), (1, -8), (2, 65), (3, NUL), (4, 4), (5, 1), (6, -1), (6, 3),
                                    (6, FAR), (8, 2), (8, -1), (21, NUL)] + at(9, LAYER_BAD) + at(17, TABLE_BAD))
    empty = list(app)
    empty[0] = empty[3] = NUL
    empty[6] = 0
    assert L.clef_kv_append(*empty) == 0
    gat = [0, *LAYER, *TABLE, P, P, 5, P, 128, P, 128, NUL]
    refused(L.clef_kv_gather, gat, at(1, LAYER_BAD) + at(9, TABLE_BAD) +
            [(0, 7), (13, NUL), (14, NUL), (15, -1), (15, FAR), (16, NUL), (16, ODD), (17, 120), (17, 132), (18, NUL), (19, 64)])
    empty = list(gat)
    empty[13] = empty[14] = empty[16] = empty[18] = NUL
    empty[15] = 0
    assert L.clef_kv_gather(*empty) == 0


def test_attention():
    L = clef.library()
    att = [P, 256, 64, 4, NUL, 4, 0, *LAYER, *TABLE, P, 0.125, 1, P, 256, 64, NUL, NUL, 0, NUL]
    refused(L.clef_kv_attention, att, [(0, NUL), (0, ODD), (1, 255), (1, -8), (2, 12), (3, -1), (3, 3), (3, FAR), (5, 3), (5, 1),
                                       (6, 9), (19, NUL), (20, float("nan")), (20, float("inf")), (22, NUL), (22, ODD),
                                       (23, 252), (23, 0), (24, 56), (25, C.c_void_p(0x10002)), (26, ODD)]
            + at(7, LAYER_BAD) + at(15, TABLE_BAD))
    empty = list(att)
    empty[0] = empty[22] = NUL
    empty[3] = 0
    assert L.clef_kv_attention(*empty) == 0
    # a long table needs a workspace
    long = list(att)
    long[15 + 1] = long[15 + 3] = 1000
    assert L.clef_kv_attention(*long) == 1 and b"workspace" in L.clef_last_error()


def test_attention_workspace():
    L = clef.library()
    n = C.c_int64(-1)

    def need(rows, ragged, seqs, hq, h, d, top):
        rc = L.clef_kv_attention_workspace(rows, ragged, seqs, hq, h, d, top, C.byref(n))
        return n.value if rc == 0 else -rc

    assert need(4, 0, 4, 8, 2, 128, 0) == 0
    assert need(0, 0, 0, 8, 2, 128, 1000) == 0
    small, large = need(4, 0, 4, 8, 2, 128, 2000), need(4, 0, 4, 8, 2, 128, 100000)
    assert 0 < small <= large
    # a shorter sequence of the call may be cut into more runs than the longest allowed one
    tops = [need(1, 0, 1, 8, 2, 64, t) for t in (100, 128, 129, 2048, 2049, 8192, 8193, 32768, 32769, 2 ** 31 - 1)]
    assert tops == sorted(tops)
    for bad in ((-1, 0, 4, 8, 2, 128, 10), (4, 0, -4, 8, 2, 128, 10), (4, 0, 4, 8, 3, 128, 10), (4, 0, 4, 8, 2, 100, 10),
                (4, 0, 4, 8, 2, 128, -1), (4, 0, 4, 8, 2, 128, FAR)):
        assert need(*bad) == -1, bad
    assert L.clef_kv_attention_workspace(4, 0, 4, 8, 2, 128, 10, NUL) == 1


POOL = [P, 4 * 2 * 16 * 64, P, 4 * 2, 6, 4, 2, 16, 64]       # with the number of planes
POOL_BAD = [(i if i < 4 else i + 1, v) for i, v in LAYER_BAD] + [(4, 0), (4, 5000)]


def test_pages():
    L = clef.library()
    res = [*TABLE, P, P, 4, 16, P, NUL]
    refused(L.clef_kv_reserve, res, TABLE_BAD + [(4, NUL), (5, NUL), (5, ODD), (6, -1), (6, FAR), (7, 24), (8, NUL), (8, ODD)])
    assert L.clef_kv_reserve(NUL, 3, 0, 3, NUL, NUL, 4, 16, NUL, NUL) == 0
    fork = [*POOL, *TABLE, P, P, P, P, 2, P, NUL]
    refused(L.clef_kv_fork, fork, POOL_BAD + at(9, TABLE_BAD) + [(13, NUL), (14, NUL), (15, NUL), (16, ODD), (17, -1),
                                                                   (17, FAR), (18, NUL), (18, ODD)])
    none = list(fork)
    none[17] = 0
    assert L.clef_kv_fork(*none) == 0
    free = [*TABLE, P, P, 4, 16, P, 2, NUL]
    refused(L.clef_kv_free, free, TABLE_BAD + [(4, NUL), (5, NUL), (6, -1), (7, 12), (8, NUL), (9, -1), (9, FAR)])
    comp = [*POOL, *TABLE, P, P, C.c_void_p(0x20000), 3, P, NUL, P, NUL]
    refused(L.clef_kv_compact, comp, POOL_BAD + at(9, TABLE_BAD) + [(13, NUL), (14, NUL), (15, NUL), (16, 2), (17, NUL),
                                                                      (18, ODD), (19, NUL)])
    inplace = list(comp)
    inplace[15], inplace[16] = P, 5                          # in place with another pitch
    assert L.clef_kv_compact(*inplace) == 1
    copy = [*POOL, P, P, 2, NUL]
    refused(L.clef_kv_copy_pages, copy, POOL_BAD + [(9, NUL), (9, ODD), (10, NUL), (11, -1), (11, FAR)])


def test_status_names():
    L = clef.library()
    assert L.clef_status_string(5) == b"CLEF_ERR_BAD_PAGE"
    assert L.clef_status_string(6) == b"CLEF_ERR_NO_PAGES"


def test_refused_tensors_need_no_gpu():
    import torch
    cpu = torch.zeros((2, 4, 2, 16, 64), dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        clef.kv_attention(torch.zeros(1, 2, 64, dtype=torch.bfloat16), cpu, torch.zeros(2, 4, 2),
                          torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        clef.w4_linear(torch.zeros(1, 128, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.uint8),
                       torch.zeros(8, 1, dtype=torch.bfloat16))


@pytest.mark.parametrize("K", [8, 128, 200, 1000])
def test_packed_layout_model(K):
    """The test model's packing and its inverse are one another's, padding included."""
    c = np.random.default_rng(K).integers(-8, 8, (3, K))
    q = w4_pack(c)
    assert np.array_equal(w4_codes(q, K), c)
    kp = q.shape[1] * 2
    assert not w4_codes(q, kp)[:, K:].any()


def test_reserve_rows():
    L = clef.library()
    res = [*TABLE, P, P, 4, 16, P, P, NUL]
    refused(L.clef_kv_reserve_rows, res, TABLE_BAD + [(4, NUL), (5, NUL), (6, -1), (7, 24), (8, NUL), (8, ODD), (9, ODD)])
    assert L.clef_kv_reserve_rows(NUL, 3, 0, 3, NUL, NUL, 4, 16, NUL, NUL, NUL) == 0


def test_attention_scale_in_log2_units():
    L = clef.library()
    att = [P, 256, 64, 4, NUL, 4, 0, *LAYER, *TABLE, P, 0.125, 1, P, 256, 64, NUL, NUL, 0, NUL]
    refused(L.clef_kv_attention, att, [(20, 3e38), (20, -3e38), (20, float("-inf"))])


def test_ragged_workspace_is_near_the_equal_rows_form():
    """With row_start the places follow the call's rows: at most those of the equal-rows form for
    sequences of a few rows, and for those of many rows a place for each row, head and run."""
    L = clef.library()
    n = C.c_int64(-1)

    def need(rows, ragged, seqs, hq, h, d, top):
        assert L.clef_kv_attention_workspace(rows, ragged, seqs, hq, h, d, top, C.byref(n)) == 0
        return n.value

    for rows, seqs, hq, h, d, top in ((64, 64, 48, 8, 128, 8192), (256, 256, 32, 8, 128, 8192), (4096, 1024, 32, 8, 128, 4096),
                                      (8, 8, 24, 4, 256, 32768), (1565, 64, 48, 8, 128, 8192), (40, 3, 8, 1, 64, 100000)):
        runs = min(16, 152 // h, -(-top // 128) // 8)
        few = 16 if top >= 8192 else 8
        if top > 16384:
            few = -(-top // 1024)
        ragged = need(rows, 1, seqs, hq, h, d, top)
        place = 4 * (d + 1)
        assert ragged <= place * rows * hq * (few + runs), (rows, seqs)
        if rows % seqs == 0 and rows // seqs * (hq // h) <= 16:
            equal = need(rows, 0, seqs, hq, h, d, top)
            assert equal <= ragged <= equal + place * min(rows * hq * runs, seqs * 152 * 256), (rows, seqs)
    assert need(1, 1, 1, 8, 2, 128, 512) == 0                   # nothing is ever cut
    # never more for more of the table
    tops = [need(100, 1, 7, 8, 2, 64, t) for t in (100, 512, 513, 1024, 1900, 2048, 8192, 8193, 40000, 10 ** 6)]
    assert tops == sorted(tops)


def test_alignment_of_row_numbers():
    L = clef.library()
    app = [P, 128, 64, P, 128, 64, 4, P, 0, *LAYER, *TABLE, P, NUL]
    refused(L.clef_kv_append, app, [(7, ODD)])
    gat = [0, *LAYER, *TABLE, P, P, 5, P, 128, P, 128, NUL]
    refused(L.clef_kv_gather, gat, [(13, ODD), (14, ODD)])
