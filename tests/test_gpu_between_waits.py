"""Waits of one cluster, or one CTA, of a call that run out while the others finish: the status says so, what the others
computed is right, and later calls are right.  (test_gpu_between_edges.py has them run out in all CTAs.)"""
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from test_gpu_fp8_block import inputs
from test_gpu_norm import values, weight

pytestmark = pytest.mark.gpu


@pytest.fixture
def only():
    """only(i): the waits of slot i (a CTA, or a cluster of pairs) of the next calls run out."""
    def force(i):
        clef.set_wait_limit_ns(20_000_000)
        clef.test_force_timeout(2 + i)

    yield force
    clef.test_force_timeout(False)
    clef.set_wait_limit_ns(1_000_000_000)
    clef.set_sm_budget(0)


def finish():
    clef.test_force_timeout(False)
    clef.set_wait_limit_ns(1_000_000_000)


@pytest.mark.parametrize("gateup", [False, True])
@pytest.mark.parametrize("m", [2, 13, 40])
@pytest.mark.parametrize("cta", [0, 1, 3])
def test_one_cta_of_a_few_rows_cluster(cta, m, gateup, only):
    """384 columns are three tiles, whose K is cut among the CTAs of a cluster: a CTA of the first gives up.
    Its peers still meet it, and the tiles of the other clusters are right."""
    f = clef.fp8_block_gateup_swiglu if gateup else clef.fp8_block_linear
    args = inputs(m, 384, 2064, 90, with_bias=True, gateup=gateup)
    want = f(*args)
    assert clef.poll_status() == 0
    only(cta)
    y = f(*args)
    assert clef.poll_status() == 4
    # (17 k-blocks: clusters of four, so that CTAs 0 to 3 are the first tile's)
    assert torch.equal(y[:, 128:], want[:, 128:])
    finish()
    assert torch.equal(f(*args), want) and clef.poll_status() == 0


@pytest.mark.parametrize("gateup,m,n,k", [(False, 2049, 264, 2064), (True, 2100, 128, 5136), (False, 4100, 384, 2064)])
@pytest.mark.parametrize("slot", [0, 1])
def test_one_cluster_of_many_rows(slot, gateup, m, n, k, only):
    """Tiles of 256 rows and all columns (or 256 of them), rows fastest, that one, two or four pairs compute: the tile of a slot."""
    f = clef.fp8_block_gateup_swiglu if gateup else clef.fp8_block_linear
    args = inputs(m, n, k, 91, with_bias=True, gateup=gateup)
    want = f(*args)
    assert clef.poll_status() == 0
    only(slot)
    y = f(*args)
    assert clef.poll_status() == 4
    keep = [i for i in range(m) if i // 256 != slot]
    assert torch.equal(y[keep], want[keep]) and torch.equal(y[:, 256:], want[:, 256:])
    finish()
    assert torch.equal(f(*args), want) and clef.poll_status() == 0


@pytest.mark.parametrize("m,n,k", [(13, 640, 2064), (2049, 264, 2064)])
def test_one_cluster_that_takes_tile_after_tile(m, n, k, only):
    """Under a budget of SMs a cluster goes from tile to tile: after its first wait ran out it still meets at every tile."""
    args = inputs(m, n, k, 92)
    want = clef.fp8_block_linear(*args)
    only(0)
    for sms in (8, 20):
        clef.set_sm_budget(sms)
        clef.fp8_block_linear(*args)
        assert clef.poll_status() == 4
    finish()
    assert torch.equal(clef.fp8_block_linear(*args), want) and clef.poll_status() == 0
    clef.set_sm_budget(0)
    assert torch.equal(clef.fp8_block_linear(*args), want) and clef.poll_status() == 0


# ---------------------------------------------------------------- rows kept ahead

@pytest.mark.parametrize("mode", ["int8_h128", "fp8_b128"])
@pytest.mark.parametrize("k", [1152, 5120])
@pytest.mark.parametrize("cta", [0, 5, 151])
def test_one_cta_of_a_norm_that_keeps_rows(cta, k, mode, only):
    """A CTA takes every so many-th row: those it left are as they were, the others right."""
    m = 1300
    x, w, r = values((m, k), 93), weight(k, 94), values((m, k), 95)
    want = clef.rms_norm_quant(x, w, mode, residual=r, residual_out=torch.empty_like(r))
    q, s = torch.full_like(want[0], 77), torch.full_like(want[1], -1.0)
    assert clef.poll_status() == 0
    only(cta)
    clef.rms_norm_quant(x, w, mode, residual=r, residual_out=torch.empty_like(r), q=q, scale=s)
    assert clef.poll_status() == 4
    left = [i for i in range(m) if not torch.equal(s[i], want[1][i])]
    step = left[1] - left[0] if len(left) > 1 else m
    assert left == list(range(cta, m, step)) and step >= 152
    rest = [i for i in range(m) if i not in left]
    assert torch.equal(q[rest], want[0][rest]) and (q[left] == 77).all() and (s[left] == -1.0).all()
    finish()
    got = clef.rms_norm_quant(x, w, mode, residual=r, residual_out=torch.empty_like(r), q=q, scale=s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and clef.poll_status() == 0
