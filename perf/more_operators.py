"""Timed cases of the operators that stand between the projections, and of the linears over block-scaled
8-bit floats: the root-mean-square norm with the residual's addition and 8-bit outputs, rotary positions,
the block-128 quantizer and the products of its codes.

Each operator has a plain form in elementary torch operations (fp32, rounded once at the end) and the
library's own call.  ``own`` chooses which of the two ``run`` computes; ``exact`` gives the values in
64 bits.  Sizes are those of the repository's decoder layers: hidden 5,120 with 6,144 query and 1,024 key
columns (48 + 8 heads of 128, or 24 + 4 of 256), feed-forward 17,408; hidden 4,096 with 12,288; the
2,048-wide linear; token counts 298, 1,502 and 24,032.
"""
import math

import torch

own = False

E4M3_TOP, INT8_TOP = 448.0, 127.0
FLT_MAX = 3.4028234663852886e38
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's residual add and norm before a 4-bit or 8-bit linear: latency
        dict(name="norm 1x5120 bf16", op="norm", m=1, k=5120, mode="bf16", y=True, residual=True),
        # a short prompt into the 2,048-wide linear: norm, rotated INT8 codes, and the product that takes them
        dict(name="norm 298x2048 int8_h128 linear", op="norm_linear", m=298, k=2048, n=2048, residual=True),
        # sixteen records of 1,502 tokens: the residual stream and the codes of the next projection in one pass
        dict(name="norm 24032x5120 fp8_b128", op="norm", m=24032, k=5120, mode="fp8_b128", y=False, residual=True),
        # a step of three answers: queries and keys of a token each
        dict(name="rotary 3x56x128", op="rotary", t=3, heads=56, spare=8, dim=128, rot=128, interleaved=False,
             theta=10000.0, factor=1.0, far=4096),
        # one prompt, a quarter of each wide head rotated in neighbouring pairs, positions of a long context
        dict(name="rotary 1502x28x256 part", op="rotary", t=1502, heads=28, spare=4, dim=256, rot=64, interleaved=True,
             theta=1000000.0, factor=16.0, far=524288),
        # sixteen packed records, whole heads
        dict(name="rotary 24032x56x128", op="rotary", t=24032, heads=56, spare=8, dim=128, rot=128, interleaved=False,
             theta=10000.0, factor=1.0, far=1502),
        # the product of gate and up of one prompt, into the down projection's codes
        dict(name="quant 1502x17408", op="quant", m=1502, k=17408, rows=1),
        # a weight, once at loading
        dict(name="quant 5120x17408 weight", op="quant", m=5120, k=17408, rows=128),
        # one token through gate and up: the largest weight read of a step
        dict(name="linear 1x5120x17408 gateup", op="linear", m=1, n=17408, k=5120, gateup=True, bias=False),
        # thirteen sequences' tokens through down, with a bias
        dict(name="linear 13x17408x5120", op="linear", m=13, n=5120, k=17408, gateup=False, bias=True),
        # one prompt through gate and up
        dict(name="linear 1502x5120x17408 gateup", op="linear", m=1502, n=17408, k=5120, gateup=True, bias=False),
        # sixteen records through the query projection
        dict(name="linear 24032x5120x6144", op="linear", m=24032, n=6144, k=5120, gateup=False, bias=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm", "norm_linear", "rotary", "rotary", "quant", "linear", "linear", "linear", "linear"])
    if op == "norm":
        mode = rng.choice(["bf16", "fp8", "fp8_h128", "fp8_b128"])
        k = 128 * log(1, 136) if mode == "fp8_h128" else 16 * log(4, 1088)
        return dict(op="norm", m=log(1, min(65536, 24032 * 5120 // k)), k=k, mode=mode, residual=rng.random() < 0.7,
                    y=mode == "bf16" or rng.random() < 0.3)
    if op == "norm_linear":
        return dict(op="norm_linear", m=log(1, 1502), k=128 * log(2, 40), n=8 * log(16, 640), residual=rng.random() < 0.7)
    if op == "rotary":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        heads = rng.choice([1, 2, 5, 8, 16, 28, 40, 56, 80])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])
        return dict(op="rotary", t=log(1, min(65536, 24032 * 56 * 128 // (heads * dim))), heads=heads, spare=rng.choice([0, 1, 8]),
                    dim=dim, rot=rot // 2 * 2, interleaved=rng.random() < 0.5, theta=rng.choice([10000.0, 500000.0, 1000000.0]),
                    factor=rng.choice([1.0, 1.0, 4.0, 16.0]), far=log(64, 1048576))
    if op == "quant":
        k = 16 * log(4, 1088)
        return dict(op="quant", m=log(1, min(34816, 34816 * 5120 // k)), k=k, rows=rng.choice([1, 1, 128]))
    k, gateup = 16 * log(8, 1088), rng.random() < 0.4
    n = 128 * log(1, 136) if gateup else 8 * log(8, 2176)
    top = 24032 * 5120 * 6144 // (k * n * (2 if gateup else 1))
    m = rng.choice([log(1, 16), log(1, max(1, min(24032, top))), log(1, max(1, min(2270, top)))])
    return dict(op="linear", m=m, n=n, k=k, gateup=gateup, bias=rng.random() < 0.5)


def _blocks(k):
    return -(-k // 128)


def work(c):
    if c["op"] in ("norm", "norm_linear"):
        m, k = c["m"], c["k"]
        b = 2.0 * m * k + 2 * k + (4.0 * m * k if c["residual"] else 0)
        if c["op"] == "norm_linear":
            n = c["n"]
            return {"bytes": b + n * k + 4 * n + 2.0 * m * n, "flops": 2.0 * m * n * k}
        if c["mode"] != "bf16":
            b += m * k + 4 * m * (_blocks(k) if c["mode"] == "fp8_b128" else 1)
        return {"bytes": b + (2.0 * m * k if c["y"] else 0), "flops": 6.0 * m * k}
    if c["op"] == "rotary":
        return {"bytes": 4.0 * c["t"] * c["heads"] * c["dim"] + 4 * c["t"] + 4 * c["rot"], "flops": 3.0 * c["t"] * c["heads"] * c["rot"]}
    if c["op"] == "quant":
        return {"bytes": 3.0 * c["m"] * c["k"] + 4 * -(-c["m"] // c["rows"]) * _blocks(c["k"]), "flops": 3.0 * c["m"] * c["k"]}
    m, n, k, wn = c["m"], c["n"], c["k"], c["n"] * (2 if c["gateup"] else 1)
    return {"bytes": 1.0 * wn * k + m * k + 4 * m * _blocks(k) + 4 * _blocks(wn) * _blocks(k) + 2.0 * m * n + (2 * wn if c["bias"] else 0),
            "flops": 2.0 * m * wn * k}


# ------------------------------------------------------------------ inputs

def _rows(shape, g, outliers=4):
    """bf16 rows with a few channels twenty times as large, as hidden states have."""
    x = torch.randn(shape, generator=g, device="cuda")
    at = torch.randint(0, shape[-1], (outliers,), generator=g, device="cuda")
    x[..., at] *= 20.0
    return x.to(torch.bfloat16)


def _frequencies(c):
    """Angle of a pair of places for one position, in 64 bits: theta ** (-2 i / rot), and where `factor` stretches
    the context (4,096 positions before), turns of 32 and more in it kept, of less than one divided by the factor,
    those between blended in proportion to their number of turns."""
    out = []
    for i in range(c["rot"] // 2):
        f = c["theta"] ** (-2.0 * i / c["rot"])
        if c["factor"] != 1.0:
            keep = min(1.0, max(0.0, (4096 * f / (2 * math.pi) - 1.0) / 31.0))
            f = f * keep + f / c["factor"] * (1.0 - keep)
        out.append(f)
    return out


def _as_turns(f):
    """Turns a position in units of 2**-64, as a signed 64-bit number."""
    u = int(round(f / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64
    return u - 2 ** 64 if u >= 2 ** 63 else u


def _padded(x, k):
    return torch.nn.functional.pad(x, (0, _blocks(k) * 128 - k)) if k % 128 else x


def _as_codes(v, top):
    return v.clamp(-top, top).to(torch.float8_e4m3fn)


def _scaled_codes(x, rows):
    """Codes and scales of x [m][k] in blocks of `rows` x 128, for inputs."""
    m, k = x.shape
    p = _padded(x.float(), k)
    if m % rows:
        p = torch.nn.functional.pad(p, (0, 0, 0, rows - m % rows))
    b = p.view(p.shape[0] // rows, rows, -1, 128)
    s = b.abs().amax(dim=(1, 3)) / E4M3_TOP
    q = _as_codes(b / torch.where(s > 0, s, torch.ones_like(s))[:, None, :, None], E4M3_TOP)
    return q.view(p.shape[0], -1)[:m, :k].contiguous(), s


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    s = dict(c=c)
    if c["op"] in ("norm", "norm_linear"):
        m, k = c["m"], c["k"]
        s["x"] = _rows((m, k), g)
        s["w"] = (1.0 + 0.2 * torch.randn(k, generator=g, device="cuda")).to(torch.bfloat16)
        s["residual"] = _rows((m, k), g) if c["residual"] else None
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
        if c["op"] == "norm_linear":
            s["qw"] = torch.randint(-127, 128, (c["n"], k), dtype=torch.int8, generator=g, device="cuda")
            s["sw"] = (0.5 + torch.rand(c["n"], generator=g, device="cuda")) / (64.0 * math.sqrt(k))
        return s
    if c["op"] == "rotary":
        # queries and keys as the packed projection leaves them, values behind
        wide = torch.randn((c["t"], (c["heads"] + c["spare"]) * c["dim"]), generator=g, device="cuda").to(torch.bfloat16)
        s["x"] = wide[:, : c["heads"] * c["dim"]].view(c["t"], c["heads"], c["dim"])
        s["pos"] = torch.randint(0, c["far"], (c["t"],), dtype=torch.int32, generator=g, device="cuda")
        f = _frequencies(c)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["turns"] = torch.tensor([_as_turns(x) for x in f], dtype=torch.int64, device="cuda")
        s["gain"] = 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0
        return s
    if c["op"] == "quant":
        s["x"] = _rows((c["m"], c["k"]), g) if c["rows"] == 1 else (
            torch.randn((c["m"], c["k"]), generator=g, device="cuda") * c["k"] ** -0.5).to(torch.bfloat16)
        return s
    wn = c["n"] * (2 if c["gateup"] else 1)
    s["qx"], s["sx"] = _scaled_codes(_rows((c["m"], c["k"]), g), 1)
    s["qw"], s["sw"] = _scaled_codes(torch.randn((wn, c["k"]), generator=g, device="cuda") * c["k"] ** -0.5, 128)
    s["bias"] = (torch.randn(wn, generator=g, device="cuda") * 0.1).to(torch.bfloat16) if c["bias"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _rotated(v):
    """Each block of 128 by the orthonormal Walsh-Hadamard butterfly."""
    m, k = v.shape
    v = v.reshape(m, k // 128, 2, 2, 2, 2, 2, 2, 2)
    for d in range(8, 1, -1):
        a, b = v.unbind(d)
        v = torch.stack((a + b, a - b), d)
    return v.reshape(m, k) * (1.0 / math.sqrt(128.0))


def _normed(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    return h, h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"].float()


def _unit(amax, top):
    """Scale and multiplier of codes whose largest is `top`."""
    r = (top / torch.where(amax > 0, amax, torch.ones_like(amax))).clamp(max=FLT_MAX)
    return amax / top, torch.where(amax > 0, r, torch.zeros_like(r))


def _plain_norm(s):
    c = s["c"]
    h, v = _normed(s)
    out = {}
    if s["residual"] is not None:
        s["sum"].copy_(h)
        out["sum"] = s["sum"]
    if c["y"]:
        out["y"] = v.to(torch.bfloat16)
    if c["mode"] == "bf16":
        return out
    if c["mode"] == "fp8_h128":
        v = _rotated(v)
    if c["mode"] == "fp8_b128":
        b = _padded(v, c["k"]).view(c["m"], -1, 128)
        scale, r = _unit(b.abs().amax(-1), E4M3_TOP)
        q = _as_codes(b * r[:, :, None], E4M3_TOP).view(c["m"], -1)[:, : c["k"]].contiguous()
    else:
        scale, r = _unit(v.abs().amax(-1), E4M3_TOP)
        q = _as_codes(v * r[:, None], E4M3_TOP)
    return out | {"q": q, "scale": scale}


def _plain_norm_linear(s):
    h, v = _normed(s)
    v = _rotated(v)
    scale, r = _unit(v.abs().amax(-1), INT8_TOP)
    q = (v * r[:, None]).round().clamp(-INT8_TOP, INT8_TOP)
    y = (q @ s["qw"].float().t()) * scale[:, None] * s["sw"]
    out = {"y": y.to(torch.bfloat16)}
    if s["residual"] is not None:
        s["sum"].copy_(h)
        out["sum"] = s["sum"]
    return out


def _plain_rotary(s):
    c = s["c"]
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["gain"]).float()[:, None], (torch.sin(angle) * s["gain"]).float()[:, None]
    x, rot = s["x"].float(), c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1).to(torch.bfloat16)


def _plain_quant(s):
    c, rows = s["c"], s["c"]["rows"]
    m, k = c["m"], c["k"]
    p = _padded(s["x"].float(), k)
    if m % rows:
        p = torch.nn.functional.pad(p, (0, 0, 0, rows - m % rows))
    b = p.view(p.shape[0] // rows, rows, -1, 128)
    scale, r = _unit(b.abs().amax(dim=(1, 3)), E4M3_TOP)
    q = _as_codes(b * r[:, None, :, None], E4M3_TOP).view(p.shape[0], -1)[:m, :k].contiguous()
    return {"q": q, "scale": scale}


def _values(q, s, rows, dtype):
    """What codes in blocks of `rows` x 128 stand for."""
    m, k = q.shape
    return q.to(dtype) * s.to(dtype).repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :k]


def _plain_linear(s):
    c = s["c"]
    y = _values(s["qx"], s["sx"], 1, torch.float32) @ _values(s["qw"], s["sw"], 128, torch.float32).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["gateup"]:
        gate, up = y.chunk(2, -1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.to(torch.bfloat16)


_PLAIN = {"norm": _plain_norm, "norm_linear": _plain_norm_linear, "rotary": _plain_rotary, "quant": _plain_quant,
          "linear": _plain_linear}


# ------------------------------------------------------------------ the library's calls

def _own_norm(s):
    c, out = s["c"], {}
    if c["mode"] == "bf16":
        y = _clef.rms_norm(s["x"], s["w"], EPS, residual=s["residual"], residual_out=s["sum"])
    else:
        y = torch.empty_like(s["x"]) if c["y"] else None
        q, scale = _clef.rms_norm_quant(s["x"], s["w"], c["mode"], EPS, residual=s["residual"], residual_out=s["sum"], y=y)
        out = {"q": q.view(torch.float8_e4m3fn), "scale": scale}
    if y is not None:
        out = {"y": y} | out
    return ({} if s["residual"] is None else {"sum": s["sum"]}) | out


def _own_norm_linear(s):
    q, scale = _clef.rms_norm_quant(s["x"], s["w"], "int8_h128", EPS, residual=s["residual"], residual_out=s["sum"])
    out = {"y": _clef.w8a8_linear(q, scale, s["qw"], s["sw"])}
    return out if s["residual"] is None else out | {"sum": s["sum"]}


def _own_rotary(s):
    return _clef.rotary(s["x"], s["pos"], s["turns"], gain=s["gain"], interleaved=s["c"]["interleaved"])


def _own_quant(s):
    q, scale = _clef.quant_fp8_block(s["x"], s["c"]["rows"])
    return {"q": q.view(torch.float8_e4m3fn), "scale": scale}


def _own_linear(s):
    call = _clef.fp8_block_gateup_swiglu if s["c"]["gateup"] else _clef.fp8_block_linear
    return call(s["qx"], s["sx"], s["qw"], s["sw"], s["bias"])


_OWN = {"norm": _own_norm, "norm_linear": _own_norm_linear, "rotary": _own_rotary, "quant": _own_quant, "linear": _own_linear}
_clef = None


def run(s):
    global _clef
    if not own:
        return _PLAIN[s["c"]["op"]](s)
    if _clef is None:
        import w8a8_quantized_projections_gb300
        _clef = w8a8_quantized_projections_gb300
    return _OWN[s["c"]["op"]](s)


# ------------------------------------------------------------------ in 64 bits

def _hadamard():
    i = torch.arange(128, device="cuda")
    both = i[:, None] & i
    odd = torch.zeros_like(both)
    for bit in range(7):
        odd ^= both >> bit & 1
    return (1.0 - 2.0 * odd.double()) / math.sqrt(128.0)


def _exact_codes(v, amax):
    """Codes before their rounding: v in units of amax / 448 (zeros for zeros)."""
    return torch.where(amax > 0, v * E4M3_TOP / torch.where(amax > 0, amax, torch.ones_like(amax)), torch.zeros_like(v))


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("norm", "norm_linear"):
        h = s["x"].double() + (0.0 if s["residual"] is None else s["residual"].double())
        v = h / torch.sqrt((h * h).sum(-1, keepdim=True) / c["k"] + EPS) * s["w"].double()
        out = {} if s["residual"] is None else {"sum": h}
        if c["op"] == "norm_linear":
            v = torch.einsum("mbi,ij->mbj", v.view(c["m"], -1, 128), _hadamard()).reshape(c["m"], -1)
            scale = v.abs().amax(-1, keepdim=True) / INT8_TOP
            q = torch.round(v / torch.where(scale > 0, scale, torch.ones_like(scale)))
            y = torch.einsum("mk,nk->mn", q, s["qw"].double()) * scale * s["sw"].double()
            return {"y": y} | out
        if c["y"]:
            out["y"] = v
        if c["mode"] == "bf16":
            return out
        if c["mode"] == "fp8_h128":
            v = torch.einsum("mbi,ij->mbj", v.view(c["m"], -1, 128), _hadamard()).reshape(c["m"], -1)
        if c["mode"] == "fp8_b128":
            amax = torch.stack([p.abs().amax(-1) for p in v.split(128, -1)], -1)
            q = _exact_codes(v, amax.repeat_interleave(128, -1)[:, : c["k"]])
        else:
            amax = v.abs().amax(-1)
            q = _exact_codes(v, amax[:, None])
        return out | {"q": q, "scale": amax / E4M3_TOP}
    if c["op"] == "rotary":
        # each pair as a complex number, turned
        rot, x = c["rot"], s["x"].double()
        first = torch.arange(rot // 2, device="cuda") * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else rot // 2)
        turn = torch.polar(torch.full((c["t"], rot // 2), s["gain"], dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * s["freq"])
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y
    if c["op"] == "quant":
        v = s["x"].double()
        amax = torch.stack([torch.stack([p.abs().amax(-1) for p in v.split(128, -1)], -1)], 0)[0]
        if c["rows"] > 1:
            amax = torch.stack([r.amax(0) for r in amax.split(c["rows"], 0)], 0)
        q = _exact_codes(v, amax.repeat_interleave(c["rows"], 0)[: c["m"]].repeat_interleave(128, 1)[:, : c["k"]])
        return {"q": q, "scale": amax / E4M3_TOP}
    x = _values(s["qx"], s["sx"], 1, torch.float64)
    wn, parts = s["qw"].shape[0], []
    for n0 in range(0, wn, 8192):
        n1 = min(wn, n0 + 8192)
        w = _values(s["qw"][n0:n1], s["sw"][n0 // 128: -(-n1 // 128)], 128, torch.float64)
        parts.append(torch.einsum("mk,nk->mn", x, w))
    y = torch.cat(parts, 1)
    if s["bias"] is not None:
        y = y + s["bias"].double()
    if c["gateup"]:
        y = y[:, : c["n"]] * torch.sigmoid(y[:, : c["n"]]) * y[:, c["n"]:]
    return y
