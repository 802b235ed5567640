"""Allowed calls at the edges of the operators between the projections: in place, pitched and far rows where CTAs keep
rows ahead, calls at once, replays, budgets, waits that run out, rows of NaN, and the largest row counts."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from between_util import bf16_off, f64, norm, norm_rel
from test_gpu_fp8_block import check_gateup, check_linear, inputs
from test_gpu_norm import MODES, values, weight
from test_gpu_rotary import check, heads, positions

pytestmark = pytest.mark.gpu
MANY = 1300          # rows from which a norm's CTAs stay and keep rows ahead (8 an SM)


def eventually(limit_ns=20_000_000):
    """Forces a wait of the next calls to run out; undone by restore()."""
    clef.set_wait_limit_ns(limit_ns)
    clef.test_force_timeout(True)


def restore():
    clef.test_force_timeout(False)
    clef.set_wait_limit_ns(1_000_000_000)


# ---------------------------------------------------------------- norms

@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("k", [640, 1152, 5120, 16384, 17408])
def test_many_rows_in_place(mode, k):
    """The sum over the residual and the result over x."""
    x, w, r = values((MANY, k), 40), weight(k, 41), values((MANY, k), 42)
    x[17] = (x[17].float() * 2.0 ** 70).to(torch.bfloat16)              # a row that is taken twice
    total, y = torch.empty_like(r), torch.empty_like(x)
    want = clef.rms_norm_quant(x, w, mode, residual=r, residual_out=total, y=y)
    xi, ri = x.clone(), r.clone()
    got = clef.rms_norm_quant(xi, w, mode, residual=ri, y=xi)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(xi, y) and torch.equal(ri, total)
    xi, ri = x.clone(), r.clone()
    assert clef.rms_norm(xi, w, residual=ri, y=xi) is xi
    assert torch.equal(xi, y) and torch.equal(ri, total)
    xi = x.clone()
    assert torch.equal(clef.rms_norm(xi, w, y=xi), clef.rms_norm(x, w)) and clef.poll_status() == 0


@pytest.mark.parametrize("k", [640, 5120, 5136])
def test_many_rows_with_pitches(k):
    wide = values((MANY, 3 * k + 24), 43)
    x, r = wide[:, :k], wide[:, k + 8:2 * k + 8]
    w = weight(k, 44)
    out = torch.full((MANY, 2 * k + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    total, y = out[:, 8:k + 8], out[:, k + 24:2 * k + 24]
    q, s = clef.rms_norm_quant(x, w, "fp8_b128", residual=r, residual_out=total, y=y)
    dense, own = r.contiguous(), torch.empty((MANY, k), dtype=torch.bfloat16, device="cuda")
    q2, s2 = clef.rms_norm_quant(x.contiguous(), w, "fp8_b128", residual=dense, y=own)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(total, dense) and torch.equal(y, own)
    for part in (out[:, :8], out[:, k + 8:k + 24], out[:, 2 * k + 24:]):
        assert (part == 7.0).all()


def test_far_rows_of_a_norm():
    """Rows past 2^32 bytes, a row at a time and kept ahead."""
    pitch = 2 ** 21 + 64
    if torch.cuda.mem_get_info()[0] < 16 * 2 ** 30:
        pytest.skip("memory")
    k = 640
    far = torch.empty(MANY * pitch, dtype=torch.bfloat16, device="cuda")
    x, y = far.as_strided((MANY, k), (pitch, 1)), far.as_strided((MANY, k), (pitch, 1), k)
    w = weight(k, 45)
    x.copy_(values((MANY, k), 46))
    assert torch.equal(clef.rms_norm(x, w, y=y), clef.rms_norm(x.contiguous(), w))
    q, s = clef.quant_fp8_block(x)
    q2, s2 = clef.quant_fp8_block(x.contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2)
    q, s = clef.quant_fp8_block(x, 128)
    q2, s2 = clef.quant_fp8_block(x.contiguous(), 128)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("m", [40, MANY])
@pytest.mark.parametrize("k", [640, 5120])
def test_rows_of_nan_stay_theirs(m, k):
    x, w = values((m, k), 47), weight(k, 48)
    plain = {mode: clef.rms_norm_quant(x, w, mode) for mode in MODES}
    y0 = clef.rms_norm(x, w)
    bad = x.clone()
    bad[3, 5], bad[m - 1, 600] = float("nan"), float("inf")
    keep = [i for i in range(m) if i not in (3, m - 1)]
    y = clef.rms_norm(bad, w)
    assert torch.equal(y[keep], y0[keep]) and y[3].isnan().all() and y[m - 1, 600].isnan()
    for mode in MODES:
        q, s = clef.rms_norm_quant(bad, w, mode)
        assert torch.equal(q[keep], plain[mode][0][keep]) and torch.equal(s[keep], plain[mode][1][keep])
        assert s[3].isnan().all()
    assert clef.poll_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_many_rows_at_once_replayed_and_under_a_budget(mode):
    """Two calls on two streams, a captured pair replayed, and few SMs: the same bits."""
    k, w = 5120, weight(5120, 49)
    xs, rs = [values((MANY, k), 50 + i) for i in range(2)], [values((MANY, k), 52 + i) for i in range(2)]
    totals = [torch.empty_like(r) for r in rs]
    want = [clef.rms_norm_quant(x, w, mode, residual=r, residual_out=torch.empty_like(r)) for x, r in zip(xs, rs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [clef.rms_norm_quant(x, w, mode, residual=r, residual_out=t, stream=s) for x, r, t, s in zip(xs, rs, totals, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    graphs, held = [], []
    for x, r, t in zip(xs, rs, totals):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(clef.rms_norm_quant(x, w, mode, residual=r, residual_out=t))
        graphs.append(g)
    for _ in range(2):
        for q, s in held:
            q.zero_(), s.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    try:
        for sms in (2, 20, 100):
            clef.set_sm_budget(sms)
            a = clef.rms_norm_quant(xs[0], w, mode, residual=rs[0], residual_out=totals[0])
            assert torch.equal(a[0], want[0][0]) and torch.equal(a[1], want[0][1])
    finally:
        clef.set_sm_budget(0)
    assert clef.poll_status() == 0


@pytest.mark.parametrize("k", [1152, 5120, 17408])
@pytest.mark.parametrize("mode", ["int8_h128", "fp8_b128"])
def test_a_norm_whose_wait_runs_out(mode, k):
    """The status says so, and later calls are right."""
    x, w, r = values((MANY, k), 56), weight(k, 57), values((MANY, k), 58)
    total, y = torch.empty_like(r), torch.empty_like(x)
    want = clef.rms_norm_quant(x, w, mode, residual=r, residual_out=total, y=y)
    assert clef.poll_status() == 0
    eventually()
    try:
        clef.rms_norm_quant(x, w, mode, residual=r, residual_out=torch.empty_like(r), y=torch.empty_like(x))
        assert clef.poll_status() == 4
    finally:
        restore()
    got = clef.rms_norm_quant(x, w, mode, residual=r, residual_out=total, y=y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and clef.poll_status() == 0


def test_without_overlapped_launches():
    x, w, r = values((MANY, 640), 59), weight(640, 60), values((MANY, 640), 61)
    args = inputs(40, 264, 640, 62)

    def run():
        return [*clef.rms_norm_quant(x, w, "fp8_b128", residual=r, residual_out=torch.empty_like(r)), *clef.quant_fp8_block(x, 128),
                clef.fp8_block_linear(*args), clef.rotary(heads(9, 4, 64, 63), positions(9, 64), clef.rotary_turns(64))]

    want = run()
    clef.set_pdl(False)
    try:
        got = run()
    finally:
        clef.set_pdl(True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_most_rows_of_short_norms():
    """More rows than 2^16 CTAs of four."""
    m, k = 300001, 16
    x, w = values((m, k), 65), weight(k, 66)
    ref = norm(x, w, 1e-6)
    assert (np.abs(f64(clef.rms_norm(x, w)) - ref) <= bf16_off(ref) + np.abs(ref) * norm_rel(k) * (1 + 2.0 ** -8)).all()


# ---------------------------------------------------------------- linears of many rows

# (from 4,097 rows on always CTA pairs; 24,100 x 2,064 in several bands of rows)
@pytest.mark.parametrize("m,n,k", [(4097, 8, 16), (4100, 264, 144), (4353, 136, 4112), (5000, 1032, 1040), (24100, 136, 2064)])
def test_linear_of_many_rows(m, n, k):
    args = inputs(m, n, k, 70, with_bias=n != 136)
    out = torch.full((m, n + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    y = clef.fp8_block_linear(*args, y=out[:, 8:n + 8])
    check_linear(y, args)
    assert (out[:, :8] == 7.0).all() and (out[:, n + 8:] == 7.0).all()
    try:
        for sms in (2, 34):
            clef.set_sm_budget(sms)
            assert torch.equal(clef.fp8_block_linear(*args), y)
    finally:
        clef.set_sm_budget(0)
    assert clef.poll_status() == 0


@pytest.mark.parametrize("m,n,k", [(4097, 128, 16), (4400, 384, 1040), (4353, 256, 4112)])
def test_gateup_of_many_rows(m, n, k):
    args = inputs(m, n, k, 71, with_bias=n == 384, gateup=True)
    out = torch.full((m, n + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    h = clef.fp8_block_gateup_swiglu(*args, h=out[:, 8:n + 8])
    check_gateup(h, args)
    assert (out[:, :8] == 7.0).all() and (out[:, n + 8:] == 7.0).all() and clef.poll_status() == 0


# (few tiles of 256 rows: two or four pairs of CTAs share one)
@pytest.mark.parametrize("gateup,m,n,k", [(False, 600, 2040, 5136), (False, 1000, 512, 4112), (False, 2049, 264, 2064), (False, 4200, 8, 8208),
                                          (True, 600, 1024, 5136), (True, 2100, 128, 5136), (True, 1281, 640, 2064)])
def test_tiles_shared_by_pairs(gateup, m, n, k):
    f, check_one = (clef.fp8_block_gateup_swiglu, check_gateup) if gateup else (clef.fp8_block_linear, check_linear)
    for with_bias in (False, True):
        args = inputs(m, n, k, 74, with_bias=with_bias, gateup=gateup)
        out = torch.full((m, n + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        y = f(*args, out[:, 8:n + 8])
        check_one(y, args)
        assert (out[:, :8] == 7.0).all() and (out[:, n + 8:] == 7.0).all()
        for sms in (0, 2, 20, 100):
            clef.set_sm_budget(sms)
            try:
                assert torch.equal(f(*args), y)
            finally:
                clef.set_sm_budget(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [f(*args) for _ in range(3)]
    for _ in range(2):
        for g in got:
            g.zero_()
        graph.replay()
        assert all(torch.equal(g, y) for g in got)
    assert clef.poll_status() == 0
    eventually()
    try:
        f(*args)
        assert clef.poll_status() == 4
        clef.set_sm_budget(20)
        f(*args)
        assert clef.poll_status() == 4
    finally:
        clef.set_sm_budget(0)
        restore()
    assert torch.equal(f(*args), y) and clef.poll_status() == 0


@pytest.mark.parametrize("gateup", [False, True])
@pytest.mark.parametrize("m", [2, 40, 4100])
def test_linears_at_once_and_waits_that_run_out(m, gateup):
    f = clef.fp8_block_gateup_swiglu if gateup else clef.fp8_block_linear
    args = [inputs(m, 384, 2064, 72 + i, gateup=gateup) for i in range(2)]
    want = [f(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [f(*a, stream=s) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert clef.poll_status() == 0
    eventually()
    try:
        f(*args[0])
        assert clef.poll_status() == 4
    finally:
        restore()
    assert torch.equal(f(*args[0]), want[0]) and clef.poll_status() == 0
    bad = args[0][1].clone()
    bad[0], bad[m - 1, 3] = float("nan"), float("inf")
    y = f(args[0][0], bad, *args[0][2:])
    assert torch.equal(y[1:m - 1], want[0][1:m - 1]) and y[0].isnan().all()


@pytest.mark.parametrize("m", [16, 300, 4200])
def test_gates_of_every_size(m):
    """Gates from -100 to 100: past the largest e^-g of fp32 and back."""
    one = torch.tensor([0x38], dtype=torch.uint8, device="cuda")               # 1.0
    qx, qw = torch.zeros((m, 128), dtype=torch.uint8, device="cuda"), torch.zeros((256, 128), dtype=torch.uint8, device="cuda")
    qx[:, 0], qw[:, 0] = one, one
    args = (qx, torch.linspace(-100, 100, m, device="cuda")[:, None].contiguous(), qw,
            torch.tensor([[1.0], [2.0 ** -16]], device="cuda"), None)
    check_gateup(clef.fp8_block_gateup_swiglu(*args), args)


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 40, 34])
def test_rotary_of_many_tokens_in_place(rot, interleaved):
    """Queries and keys of packed rows, one after the other on the same rows; two streams; replays."""
    t, turns = 3001, clef.rotary_turns(rot)
    wide = heads(t, 12, 128, 80, spare=3).contiguous()
    packed = torch.randn((t, 12 * 128 + 64), generator=torch.Generator().manual_seed(81)).to(torch.bfloat16).cuda()
    before = packed.clone()
    pos = positions(t, 82)
    q, k = (packed[:, a * 128:b * 128].unflatten(1, (b - a, 128)) for a, b in ((0, 8), (8, 10)))
    want = [clef.rotary(v.contiguous(), pos, turns, interleaved=interleaved) for v in (q, k)]
    check(want[0], q, pos, turns, interleaved=interleaved)
    torch.cuda.synchronize()
    for v, s in zip((q, k), (torch.cuda.Stream(), torch.cuda.Stream())):
        clef.rotary(v, pos, turns, interleaved=interleaved, out=v, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(packed[:, 1280:], before[:, 1280:])
    out = torch.empty_like(wide)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clef.rotary(wide, pos, turns, interleaved=interleaved, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, clef.rotary(wide, pos, turns, interleaved=interleaved))
