"""What needs no GPU of the operators between the projections: refusals of the C ABI, and the
tables of rotary positions."""
import ctypes as C
import math

import pytest

import w8a8_quantized_projections_gb300 as clef

P = C.c_void_p(0x10000)          # 16-byte aligned, never dereferenced
ODD = C.c_void_p(0x10008)
Z = C.c_void_p(None)
NORM = dict(x=P, ldx=256, r=P, ldr=256, w=P, M=4, K=256, eps=1e-6, ro=P, ldro=256, y=P, ldy=256)
ORDER = ("x", "ldx", "r", "ldr", "w", "M", "K", "eps", "ro", "ldro", "y", "ldy")


@pytest.mark.parametrize("bad", [dict(x=Z), dict(x=ODD), dict(w=Z), dict(w=ODD), dict(ldx=248), dict(ldx=260), dict(ldr=8), dict(ldro=250),
                                 dict(ro=Z), dict(r=Z), dict(y=Z), dict(y=ODD), dict(ldy=0), dict(M=-1), dict(M=2 ** 31), dict(K=0),
                                 dict(K=24, ldx=256), dict(K=32784, ldx=32784, ldr=32784, ldro=32784, ldy=32784), dict(eps=0.0),
                                 dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf)])
def test_norm_refusals(bad):
    a = NORM | bad
    assert clef.library().clef_rms_norm(*[a[n] for n in ORDER], Z) == 1


@pytest.mark.parametrize("mode,bad", [(-1, {}), (4, {}), (0, dict(K=144, ldx=144)), (2, dict(K=144, ldx=144)), (3, dict(K=120, ldx=120)),
                                      (0, dict(q=Z)), (0, dict(q=ODD)), (1, dict(scale=Z)), (1, dict(scale=C.c_void_p(0x10002))),
                                      (3, dict(y=ODD)), (3, dict(r=Z))])
def test_norm_quant_refusals(mode, bad):
    a = NORM | dict(q=P, scale=P) | bad
    head = [a[n] for n in ("x", "ldx", "r", "ldr", "w", "M", "K", "eps")]
    assert clef.library().clef_rms_norm_quant(*head, mode, a["ro"], a["ldro"], a["y"], a["ldy"], a["q"], a["scale"], Z) == 1


@pytest.mark.parametrize("args", [(Z, 4, 256, 256, 1, P, P), (P, 4, 256, 256, 2, P, P), (P, 4, 256, 256, 0, P, P), (P, -1, 256, 256, 1, P, P),
                                  (P, 4, 250, 256, 1, P, P), (P, 4, 256, 128, 1, P, P), (P, 4, 256, 260, 1, P, P), (ODD, 4, 256, 256, 1, P, P),
                                  (P, 4, 256, 256, 128, ODD, P), (P, 4, 256, 256, 128, P, C.c_void_p(0x10001)),
                                  (P, 4, 65552, 65552, 1, P, P)])
def test_quant_block_refusals(args):
    assert clef.library().clef_quant_fp8_block(*args, Z) == 1


ROT = dict(x=P, ldx=512, ldh=128, t=3, heads=4, dim=128, rot=128, inter=0, pos=P, turns=P, gain=1.0, out=C.c_void_p(0x90000), ldo=512, ldoh=128)


@pytest.mark.parametrize("bad", [dict(x=Z), dict(x=ODD), dict(out=ODD), dict(pos=Z), dict(turns=Z), dict(turns=C.c_void_p(0x10004)),
                                 dict(pos=C.c_void_p(0x10002)), dict(t=-1), dict(t=2 ** 31), dict(heads=0), dict(heads=1025), dict(dim=124),
                                 dict(dim=0), dict(dim=1032, ldx=8192, ldh=1032, ldo=8192, ldoh=1032), dict(rot=0), dict(rot=3), dict(rot=130),
                                 dict(ldx=100), dict(ldh=64), dict(ldo=516), dict(ldoh=0), dict(gain=math.inf), dict(gain=math.nan),
                                 dict(out=P, ldo=1024)])
def test_rotary_refusals(bad):
    assert clef.library().clef_rotary(*(ROT | bad).values(), Z) == 1


def test_empty_calls_need_no_pointers():
    L = clef.library()
    assert L.clef_rms_norm(Z, 256, Z, 0, Z, 0, 256, 1e-6, Z, 0, Z, 0, Z) == 0
    assert L.clef_quant_fp8_block(Z, 0, 256, 256, 1, Z, Z, Z) == 0
    assert L.clef_rotary(*(ROT | dict(t=0, x=Z, out=Z, pos=Z)).values(), Z) == 0


# ---------------------------------------------------------------- tables

def frequencies(t):
    return [(x % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for x in t.tolist()]


@pytest.mark.parametrize("rot,theta", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (34, 1e6)])
def test_turns(rot, theta):
    t = clef.rotary_turns(rot, theta, device="cpu")
    assert t.shape == (rot // 2,)
    for i, f in enumerate(frequencies(t)):
        assert abs(f - theta ** (-2 * i / rot)) <= 2.0 ** -45 * f + 2.0 ** -62
    assert frequencies(t)[0] == pytest.approx(1.0, rel=1e-14)


def test_scaled_turns():
    base, rot, s = frequencies(clef.rotary_turns(64, device="cpu")), 64, 8.0
    linear = frequencies(clef.rotary_turns(rot, scaling="linear", factor=s, device="cpu"))
    assert all(a == pytest.approx(b / s, rel=1e-12) for a, b in zip(linear, base))
    theta = frequencies(clef.rotary_turns(rot, scaling="theta", factor=s, device="cpu"))
    assert theta[0] == pytest.approx(base[0], rel=1e-12) and theta[-1] == pytest.approx(base[-1] / s, rel=1e-12)
    parts = frequencies(clef.rotary_turns(rot, scaling="by_parts", factor=s, original=2048, slow=1, fast=32, device="cpu"))
    for a, b in zip(parts, base):
        n = b * 2048 / (2 * math.pi)
        if n >= 32:
            assert a == pytest.approx(b, rel=1e-12)
        elif n <= 1:
            assert a == pytest.approx(b / s, rel=1e-12)
        else:
            keep = (n - 1) / 31
            assert a == pytest.approx(b * keep + b / s * (1 - keep), rel=1e-12)
    assert parts[0] == pytest.approx(base[0]) and parts[-1] == pytest.approx(base[-1] / s)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=8, scaling="other"), dict(rot=8, theta=0.0), dict(rot=8, factor=0.5),
                                dict(rot=8, slow=4, fast=4), dict(rot=2, scaling="theta", factor=2.0), dict(rot=8, theta=math.inf)])
def test_turns_refusals(kw):
    with pytest.raises(ValueError):
        clef.rotary_turns(**kw, device="cpu")


# ---------------------------------------------------------------- block linears

LIN = dict(qx=P, sx=P, qw=P, sw=P, bias=Z, M=4, N=256, K=512, y=P, ldy=256)


@pytest.mark.parametrize("name", ["clef_fp8_block_linear", "clef_fp8_block_gateup_swiglu"])
@pytest.mark.parametrize("bad", [dict(qx=Z), dict(qx=ODD), dict(sx=Z), dict(sx=C.c_void_p(0x10002)), dict(qw=ODD), dict(sw=Z),
                                 dict(sw=C.c_void_p(0x10001)), dict(bias=ODD), dict(M=-1), dict(M=2 ** 31), dict(N=0), dict(N=4, ldy=8),
                                 dict(N=2 ** 30), dict(K=0), dict(K=40), dict(K=65552), dict(y=Z), dict(y=ODD), dict(ldy=248), dict(ldy=260)])
def test_block_linear_refusals(name, bad):
    assert getattr(clef.library(), name)(*(LIN | bad).values(), Z) == 1


def test_gateup_needs_whole_blocks():
    L = clef.library()
    assert L.clef_fp8_block_gateup_swiglu(*(LIN | dict(N=136, ldy=136)).values(), Z) == 1
    assert L.clef_fp8_block_linear(*(LIN | dict(M=0, qx=Z, sx=Z, y=Z)).values(), Z) == 0
