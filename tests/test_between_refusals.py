"""Calls of the operators between the projections that are refused: in place with another pitch."""
import ctypes as C

import pytest

import w8a8_quantized_projections_gb300 as clef

P, Q, R = (C.c_void_p(0x10000 * i) for i in (1, 2, 3))          # 16-byte aligned, never dereferenced
Z = C.c_void_p(None)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("y,ldy,out,ldro", [(P, 512, R, 256), (P, 264, R, 256), (Q, 256, R, 512), (P, 512, R, 512)])
def test_in_place_with_another_pitch(y, ldy, out, ldro, quant):
    """Rows of the result over rows that have not been read."""
    L = clef.library()
    a = (P, 256, R, 256, Q, 4, 256, 1e-6)                        # x, its pitch, residual, its pitch, w, rows, columns, eps
    rc = L.clef_rms_norm_quant(*a, 3, out, ldro, y, ldy, Q, Q, Z) if quant else L.clef_rms_norm(*a, out, ldro, y, ldy, Z)
    assert rc == 1
    assert b"pitches must agree" in L.clef_last_error()

