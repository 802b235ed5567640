"""Norms of short rows by more than 65,536 CTAs: the last rows against 64 bits, all of them against calls of fewer rows."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from between_util import bf16_off, f64, norm, norm_rel
from test_gpu_norm import check_quant, weight

pytestmark = pytest.mark.gpu


# rows a CTA: 16 of up to 128 values, 8 of up to 256, 4 of up to 512 (and of up to 1,024 where none are rotated)
@pytest.mark.parametrize("k,per", [(16, 16), (128, 16), (144, 8), (272, 4), (384, 4)])
def test_more_ctas_than_16_bits(k, per):
    m = 65536 * per + 3
    g = torch.Generator(device="cuda").manual_seed(k)
    x = torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16)
    w = weight(k, 1)
    y = clef.rms_norm(x, w)
    tail = x[-1000:].contiguous()
    ref = norm(tail, w, 1e-6)
    assert (np.abs(f64(y[-1000:]) - ref) <= bf16_off(ref) + norm_rel(k) * np.abs(ref)).all()
    q, s = clef.rms_norm_quant(x, w, "fp8_b128")
    check_quant(q[-1000:], s[-1000:], "fp8_b128", ref, norm_rel(k))
    for a in range(0, m, 300001):
        part = x[a:a + 300001]
        assert torch.equal(clef.rms_norm(part, w), y[a:a + 300001])
        qp, sp = clef.rms_norm_quant(part, w, "fp8_b128")
        assert torch.equal(qp, q[a:a + 300001]) and torch.equal(sp, s[a:a + 300001])
    assert clef.poll_status() == 0
