"""Timed cases of the single-token operators: 4-bit linears, the 8-bit paged cache and the
attention that reads it, and the page bookkeeping.

Each operator has a plain form in elementary torch operations (fp32, rounded once at the end) and the
library's own call.  ``own`` chooses which of the two ``run`` computes; ``exact`` gives the values in
64 bits.  The head shapes are those that the projections of the repository's decoder layers allow:
6,144 query and 1,024 key/value columns are 48/8 heads of 128 or 24/4 of 256, 4,096 query columns are
32/8 heads of 128.
"""
import math

import torch

own = False

INT8_TOP, E4M3_TOP = 127.0, 448.0
FLT_MAX = 3.4028234663852886e38


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through the o projection of the 27B-shaped layer: the smallest weight read of a step
        dict(name="w4 1x6144x5120 g128", op="w4", m=1, n=5120, k=6144, group=128, bias=False),
        # one token through the packed gate/up weight: the largest weight read of a step
        dict(name="w4 1x5120x34816 g64", op="w4", m=1, n=34816, k=5120, group=64, bias=False),
        # thirteen sequences' tokens through down, with the finest groups and a bias
        dict(name="w4 13x17408x5120 g32", op="w4", m=13, n=5120, k=17408, group=32, bias=True),
        # one sequence with a short prompt: latency
        dict(name="attend 1x298 int8", op="attend", b=1, n=1, lo=298, hi=298, hq=48, hkv=8, d=128, page=64,
             kind="int8", causal=True),
        # a serving batch of ragged lengths, one token each
        dict(name="attend 64x512-8192 int8", op="attend", b=64, n=1, lo=512, hi=8192, hq=48, hkv=8, d=128, page=64,
             kind="int8", causal=True),
        # few sequences with a long context, wide heads
        dict(name="attend 3x32768 e4m3 d256", op="attend", b=3, n=1, lo=30011, hi=32768, hq=24, hkv=4, d=256, page=128,
             kind="e4m3", causal=True),
        # eight questions of 48 tokens asked of records of about 1,502 tokens
        dict(name="attend 8x48 of 1550 int8 d256", op="attend", b=8, n=48, lo=1550, hi=1550, hq=24, hkv=4, d=256, page=32,
             kind="int8", causal=True),
        # a whole record of 2,270 tokens attends to itself
        dict(name="attend 1x2270 of 2270 e4m3", op="attend", b=1, n=2270, lo=2270, hi=2270, hq=32, hkv=8, d=128, page=64,
             kind="e4m3", causal=True),
        # a serving step's new tokens, one a sequence
        dict(name="append 64x1 int8", op="append", b=64, n=1, lo=512, hi=8192, h=8, d=128, page=64, kind="int8"),
        # sixteen records of 1,502 tokens written at once
        dict(name="append 16x1502 e4m3", op="append", b=16, n=1502, lo=1502, hi=1550, h=8, d=128, page=64, kind="e4m3"),
        # two records' pages shared by four questions each, that grow by 48 tokens and are dropped again
        dict(name="fork 8 of 1502", op="fork", b=24, forks=8, grow=48, lo=1400, hi=1600, pages=2048, planes=16, h=8,
             d=128, page=64, kind="int8"),
        # a half-empty pool moved together
        dict(name="compact 1024 pages", op="compact", b=40, live=0.5, pages=1024, planes=16, h=8, d=128, page=64,
             kind="int8"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["w4", "w4", "attend", "attend", "attend", "append", "pages"])
    kind = rng.choice(["int8", "e4m3"])
    if op == "w4":
        k = 8 * log(32, 2176)
        n = log(64, min(34816, 34816 * 5120 // k))
        return dict(op="w4", m=log(1, 16), n=n, k=k, group=rng.choice([32, 64, 128]), bias=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128, 128, 256])
    if op == "attend":
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 3, 4, 6, 8, 16])
        while hkv * g > 64:
            g //= 2
        b, hi = log(1, 64), log(64, 32768)
        n = 1 if rng.random() < 0.6 else log(2, 2270)
        # no more work than the largest listed cases: 64 sequences of 8,192 tokens, or 2,270 rows of 2,270
        hi = max(16, min(hi, 64 * 8192 * 8 * 128 // (4 * b * hkv * d)))
        n = min(n, hi, max(1, 2270 * 2270 * 32 * 128 // (b * hi * hkv * g * d)))
        lo = max(n, int(hi * rng.uniform(0.05, 1.0)), 1)
        return dict(op="attend", b=b, n=n, lo=lo, hi=max(lo, hi), hq=hkv * g, hkv=hkv, d=d, page=page, kind=kind,
                    causal=rng.random() < 0.8)
    if op == "append":
        h = rng.choice([1, 2, 4, 8])
        b = log(1, 64)
        n = log(1, max(2, 16 * 1502 * 8 * 128 // (b * h * d)))
        n = min(n, 4096)
        lo = n + log(1, 2048) - 1
        return dict(op="append", b=b, n=n, lo=lo, hi=lo + log(1, 1024), h=h, d=d, page=page, kind=kind)
    h, planes = rng.choice([1, 4, 8]), 2 * log(1, 8)
    pages = min(4096, 1024 * 64 * 8 * 128 * 16 // (page * h * d * planes))
    pages = log(96, max(97, pages))
    if rng.random() < 0.5:
        return dict(op="compact", b=log(1, min(64, pages // 4)), live=round(rng.uniform(0.1, 0.9), 3), pages=pages,
                    planes=planes, h=h, d=d, page=page, kind=kind)
    b, forks = log(1, 8), log(1, 16)
    each = max(1, pages // (2 * (b + forks)))         # pages a sequence may hold
    hi = each * page - rng.randrange(page)
    return dict(op="fork", b=b + forks, forks=forks, grow=log(1, page), lo=max(1, hi // 2), hi=hi, pages=pages,
                planes=planes, h=h, d=d, page=page, kind=kind)


def work(c):
    if c["op"] == "w4":
        kp = -(-c["k"] // 128) * 128
        return {"bytes": c["n"] * kp / 2 + 2 * c["n"] * kp / c["group"] + 2 * c["m"] * (c["k"] + c["n"])
                + 2 * c["n"] * c["bias"], "flops": 2.0 * c["m"] * c["n"] * c["k"]}
    if c["op"] == "attend":
        lens, n = _lengths(c), c["n"]
        t = c["b"] * n
        pages = sum(-(-x // c["page"]) for x in lens)
        kv = sum(lens) * 2 * c["hkv"] * c["d"] + 8 * c["hkv"] * pages
        pairs = sum(n * x - (n * (n - 1) // 2 if c["causal"] else 0) for x in lens)
        return {"bytes": kv + 4 * pages + 4 * c["b"] + 4.0 * t * c["hq"] * c["d"], "flops": 4.0 * pairs * c["hq"] * c["d"]}
    row = c["h"] * c["d"]
    if c["op"] == "append":
        t, touched, held = c["b"] * c["n"], 0, 0
        for x in _lengths(c):
            first = (x - c["n"]) // c["page"]
            touched += (x - 1) // c["page"] - first + 1
            held += (x - c["n"]) - first * c["page"]
        # new rows read in 2 bytes and written as codes; then codes read back and values written in 2 bytes
        return {"bytes": t * row * 2 * 3.0 + (t + held) * row * 2 * 3.0 + touched * c["h"] * 16 + (t + held) * 8,
                "flops": 8.0 * t * row}
    page_bytes = c["planes"] * (c["page"] * row + 4 * c["h"])
    if c["op"] == "fork":
        lens = _lengths(c)[: c["b"] - c["forks"]]
        per = [lens[i // 4 % len(lens)] for i in range(c["forks"])]
        tails = sum(1 for x in per if x % c["page"])
        held = sum(-(-x // c["page"]) for x in per)
        return {"bytes": 2.0 * tails * page_bytes + 4 * c["pages"] + 24 * held + 16 * c["b"], "flops": 0}
    live, moves = _plan_pages(c)[1:]
    return {"bytes": 2.0 * moves * page_bytes + 8 * c["pages"] + 8 * live, "flops": 0}


# ------------------------------------------------------------------ inputs

def _mix(i):
    """A fixed pseudo-random number of [0, 1) for place i."""
    x = (i * 0x9E3779B97F4A7C15 + 0x632BE59BD9B4E019) & (2 ** 64 - 1)
    x = ((x ^ (x >> 30)) * 0xBF58476D1CE4E5B9) & (2 ** 64 - 1)
    x = ((x ^ (x >> 27)) * 0x94D049BB133111EB) & (2 ** 64 - 1)
    return (x ^ (x >> 31)) / 2 ** 64


def _lengths(c):
    """Lengths of a case's sequences (the same for every seed), spread over [lo, hi]."""
    r = [int(round(c["lo"] * (c["hi"] / c["lo"]) ** _mix(i))) for i in range(c["b"])]
    r[0] = c["hi"]
    return r


def _plan_pages(c):
    """compact: the pages held by the case's sequences, their number and how many of them have to move."""
    n, want = c["pages"], max(c["b"], int(c["pages"] * c["live"]))
    order = sorted(range(n), key=lambda p: _mix(p + 7919))
    held = sorted(order[:want])
    return held, len(held), sum(1 for p in held if p >= len(held))


def _top(kind):
    return INT8_TOP if kind == "int8" else E4M3_TOP


def _random_codes(shape, kind, g):
    """Codes as a quantized cache holds them: normal values, the block's largest near the top code."""
    x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0, 0.28, generator=g)
    x = x.clamp_(-1, 1).mul_(_top(kind))
    return x.round_().to(torch.int8) if kind == "int8" else x.to(torch.float8_e4m3fn).view(torch.uint8)


def _rows(shape, g, outliers=4):
    """bf16 rows with a few channels twenty times as large, as hidden states have."""
    x = torch.randn(shape, generator=g, device="cuda")
    at = torch.randint(0, shape[-1], (outliers,), generator=g, device="cuda")
    x[..., at] *= 20.0
    return x.to(torch.bfloat16)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    if c["op"] == "w4":
        kp = -(-c["k"] // 128) * 128
        qw = torch.randint(0, 256, (c["n"], kp // 2), dtype=torch.uint8, generator=g, device="cuda")
        if kp > c["k"]:                       # columns past k hold the code of zero
            codes = _unpack(qw)
            codes[:, c["k"]:] = 0
            qw = _pack(codes)
        sw = (torch.rand((c["n"], kp // c["group"]), generator=g, device="cuda") * 0.006 + 0.002).to(torch.bfloat16)
        bias = (torch.randn(c["n"], generator=g, device="cuda") * 0.01).to(torch.bfloat16) if c["bias"] else None
        return dict(c=c, x=_rows((c["m"], c["k"]), g, 8), qw=qw, sw=sw, bias=bias)
    P, D = c["page"], c["d"]
    if c["op"] in ("attend", "append"):
        H = c["hkv"] if c["op"] == "attend" else c["h"]
        lens = _lengths(c)
        counts = [-(-x // P) for x in lens]
        width, pages = max(counts), sum(counts) + 3
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((c["b"], width), -1, dtype=torch.int32)
        flat, at = perm.cpu(), 0
        for i, k in enumerate(counts):
            table[i, :k] = flat[at:at + k]
            at += k
        codes = _random_codes((2, pages, H, P, D), c["kind"], g)
        scales = (torch.rand((2, pages, H), generator=g, device="cuda") * 2.0 + 2.5) / _top(c["kind"])
        s = dict(c=c, codes=codes, scales=scales, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        t = c["b"] * c["n"]
        if c["op"] == "attend":
            # queries as the packed projection leaves them: a column block of wider rows
            wide = torch.randn((t, (c["hq"] + 2 * H) * D), generator=g, device="cuda").to(torch.bfloat16)
            s["q"] = wide[:, : c["hq"] * D].view(t, c["hq"], D)
            return s
        wide = _rows((t, 2 * H * D), g)
        s["k"], s["v"] = wide[:, : H * D].view(t, H, D), wide[:, H * D:].view(t, H, D)
        first = [(x - c["n"]) // P * P for x in lens]
        s["seq"] = torch.cat([torch.full((x - f,), i, dtype=torch.int32) for i, (x, f) in enumerate(zip(lens, first))]).cuda()
        s["pos"] = torch.cat([torch.arange(f, x, dtype=torch.int32) for x, f in zip(lens, first)]).cuda()
        return s
    # pages: a pool of `planes` planes (each layer's keys, then its values) with one table
    codes = torch.randint(-127, 128, (c["planes"], c["pages"], c["h"], P, D), dtype=torch.int8, generator=g, device="cuda")
    if c["kind"] == "e4m3":
        codes = codes.view(torch.uint8)
    scales = torch.rand((c["planes"], c["pages"], c["h"]), generator=g, device="cuda") + 0.5
    refs = torch.zeros(c["pages"], dtype=torch.int32)
    if c["op"] == "fork":
        own_n = c["b"] - c["forks"]
        lens = _lengths(c)[:own_n]
        counts = [-(-x // P) for x in lens]
        width = -(-(max(lens) + c["grow"]) // P)
        perm = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32).cpu()
        table, at = torch.full((c["b"], width), -1, dtype=torch.int32), 0
        for i, k in enumerate(counts):
            table[i, :k] = perm[at:at + k]
            at += k
        refs[perm[:at].long()] = 1
        src = torch.tensor([i // 4 % own_n for i in range(c["forks"])], dtype=torch.int32)
        dst = torch.arange(own_n, c["b"], dtype=torch.int32)
        grow = torch.zeros(c["b"], dtype=torch.int32)
        grow[own_n:] = c["grow"]
        return dict(c=c, codes=codes, scales=scales, refs=refs.cuda(), table=table.cuda(), src=src.cuda(), dst=dst.cuda(),
                    grow=grow.cuda(), lens=torch.tensor(lens + [0] * c["forks"], dtype=torch.int32, device="cuda"))
    held, live, _ = _plan_pages(c)
    perm = torch.tensor(held, dtype=torch.int32)[torch.randperm(live, generator=g, device="cuda").cpu()]
    refs[perm.long()] = 1
    cuts = [live * i // c["b"] for i in range(c["b"] + 1)]
    counts = [y - x for x, y in zip(cuts, cuts[1:])]
    table = torch.full((c["b"], max(counts)), -1, dtype=torch.int32)
    for i, k in enumerate(counts):
        table[i, :k] = perm[cuts[i]:cuts[i + 1]]
    lens = [max(0, k * P - int(P * _mix(i))) for i, k in enumerate(counts)]
    return dict(c=c, codes=codes, scales=scales, refs=refs.cuda(), table=table.cuda(),
                table_out=torch.full_like(table, -1).cuda(), refs_out=torch.zeros_like(refs).cuda(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ plain forms

_OFFSET = [0, 4, 1, 5, 2, 6, 3, 7]        # nibble of a word that holds the o-th of its eight codes


def _unpack(qw):
    """Signed codes [n][kp] of packed 4-bit rows."""
    n, kb = qw.shape[0], qw.shape[1] // 64
    w = qw.view(torch.int32).view(n, kb, 4, 4, 1)
    shift = 4 * torch.tensor(_OFFSET, dtype=torch.int32, device=qw.device)
    codes = ((w >> shift) & 15) - 8                                   # [n][kb][t][j][8]
    return codes.permute(0, 1, 3, 2, 4).reshape(n, kb * 128).to(torch.int8)


def _pack(codes):
    n, kb = codes.shape[0], codes.shape[1] // 128
    u = (codes.to(torch.int32) + 8).view(n, kb, 4, 4, 8).permute(0, 1, 3, 2, 4)
    shift = 4 * torch.tensor(_OFFSET, dtype=torch.int32, device=codes.device)
    w = (u.to(torch.int64) << shift.to(torch.int64)).sum(-1)
    w = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
    return w.contiguous().view(torch.uint8).view(n, kb * 64)


def _values(codes, kind):
    return codes.to(torch.float32) if kind == "int8" else codes.view(torch.float8_e4m3fn).to(torch.float32)


def _codes(v, kind):
    if kind == "int8":
        return v.round().clamp(-INT8_TOP, INT8_TOP).to(torch.int8)
    return v.clamp(-E4M3_TOP, E4M3_TOP).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_w4(s):
    c, x = s["c"], s["x"].float()
    codes = _unpack(s["qw"]).float()
    w = (codes.view(c["n"], -1, c["group"]) * s["sw"].float()[:, :, None]).view(c["n"], -1)[:, : c["k"]]
    y = x @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(torch.bfloat16)


def _plain_attend(s):
    c = s["c"]
    b, n, hk, d, P = c["b"], c["n"], c["hkv"], c["d"], c["page"]
    g, top = c["hq"] // hk, s["table"].shape[1] * P
    at = s["table"].clamp(min=0).long()
    kv = _values(s["codes"][:, at], c["kind"]) * s["scales"][:, at][..., None, None]   # [2][b][pages][h][P][d]
    kv = kv.permute(0, 1, 3, 2, 4, 5).reshape(2, b, hk, top, d)
    q = s["q"].float().view(b, n, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, n * g, d)
    a = (q @ kv[0].transpose(-1, -2)) / math.sqrt(d)
    lens = s["lens"].long()
    j = torch.arange(top, device=q.device)
    end = lens[:, None].expand(b, n)
    if c["causal"]:
        end = end - n + 1 + torch.arange(n, device=q.device)
    seen = (j < end[:, :, None])[:, None, :, None, :]                                   # [b][1][n][1][top]
    a = a.view(b, hk, n, g, top).masked_fill(~seen, float("-inf"))
    m = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    z = e.sum(-1, keepdim=True)
    p = (e / torch.where(z > 0, z, torch.ones_like(z))).view(b, hk, n * g, top)
    o = p @ kv[1]
    return o.view(b, hk, n, g, d).permute(0, 2, 1, 3, 4).reshape(b * n, c["hq"], d).to(torch.bfloat16)


def _plain_append(s):
    c = s["c"]
    b, n, h, d, P = c["b"], c["n"], c["h"], c["d"], c["page"]
    codes, scales, lens = s["codes"], s["scales"], s["lens"].long()
    x = torch.stack([s["k"], s["v"]]).float().view(2, b, n, h, d)
    start = lens - n
    first = start // P
    pos = start[:, None] + torch.arange(n, device=x.device)                # [b][n]
    slot = pos // P - first[:, None]
    width = (n + P - 2) // P + 1
    amax = torch.zeros((2, b, width, h), device=x.device).scatter_reduce_(
        2, slot[None, :, :, None].expand(2, b, n, h), x.abs().amax(-1), "amax")
    held = start - first * P                                               # tokens already in the first page
    spot = (first[:, None] + torch.arange(width, device=x.device)).clamp(max=s["table"].shape[1] - 1)
    page = torch.gather(s["table"].long(), 1, spot)                        # [b][width]
    old = torch.zeros((2, b, width, h), device=x.device)
    old[:, :, 0] = torch.where((held > 0)[None, :, None], scales[:, page[:, 0]], old[:, :, 0])
    new = torch.maximum(old, amax / _top(c["kind"]))
    inv = torch.where(new > 0, (1.0 / new).clamp(max=FLT_MAX), torch.zeros_like(new))
    # the tokens already there, in the new scale
    ratio = torch.where(new[:, :, 0] > 0, old[:, :, 0] / new[:, :, 0], torch.ones_like(new[:, :, 0]))
    was = codes[:, page[:, 0]]                                             # [2][b][h][P][d]
    now = _codes(_values(was, c["kind"]) * ratio[..., None, None], c["kind"])
    keep = (torch.arange(P, device=x.device) < held[:, None])[None, :, None, :, None] & (ratio < 1)[..., None, None]
    codes[:, page[:, 0]] = torch.where(keep, now, was)
    # the new tokens
    q = _codes(x * torch.gather(inv, 2, slot[None, :, :, None].expand(2, b, n, h))[..., None], c["kind"])
    at = torch.gather(page, 1, slot)
    codes.permute(1, 3, 0, 2, 4)[at.reshape(-1), (pos % P).reshape(-1)] = q.permute(1, 2, 0, 3, 4).reshape(b * n, 2, h, d)
    touched = slot[:, -1:] >= torch.arange(width, device=x.device)
    spare = scales.shape[1]                                                # a row of its own for untouched slots
    grown = torch.cat([scales, torch.zeros_like(scales[:, :1])], 1)
    grown[:, torch.where(touched, page, torch.full_like(page, spare)).reshape(-1)] = new.reshape(2, -1, h)
    scales.copy_(grown[:, :spare])
    # what the cache now stands for, from the first touched page of each sequence on
    seq, p = s["seq"].long(), s["pos"].long()
    at = s["table"].long()[seq, p // P]
    out = _values(codes.permute(1, 3, 0, 2, 4)[at, p % P], c["kind"]) * scales[:, at].permute(1, 0, 2)[..., None]
    k, v = out.to(torch.bfloat16).unbind(1)
    return {"k": k, "v": v, "scales": scales}


def _lowest_free(refs, n):
    return torch.argsort((refs > 0).to(torch.int8), stable=True)[:n]


def _plain_fork(s):
    c = s["c"]
    P, table, lens, refs, codes, scales = c["page"], s["table"], s["lens"], s["refs"], s["codes"], s["scales"]
    src, dst, n = s["src"].long(), s["dst"].long(), c["forks"]
    col = torch.arange(table.shape[1], device=table.device)
    # fork: whole pages shared, a part-filled last page copied to the lowest free page
    size = lens[src].long()
    count, full = (size + P - 1) // P, size // P
    tail = count > full
    rank = torch.cumsum(tail.long(), 0) - 1
    fresh = _lowest_free(refs, n)[rank.clamp(min=0)]
    rows = torch.where(col < count[:, None], table[src], table[dst])
    last = torch.gather(rows, 1, full.clamp(max=table.shape[1] - 1)[:, None]).long()[:, 0]
    to = torch.where(tail, fresh, last)
    kept = torch.where(tail, last, to)
    codes[:, to] = codes[:, kept]
    scales[:, to] = scales[:, kept]
    is_tail = tail[:, None] & (col == full[:, None])
    table[dst] = torch.where(is_tail, fresh[:, None].to(torch.int32), rows)
    shared = torch.where(col < full[:, None], rows, torch.full_like(rows, c["pages"])).long().reshape(-1)
    more = torch.zeros(c["pages"] + 1, dtype=torch.int32, device=refs.device)
    more.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    more.index_add_(0, torch.where(tail, fresh, torch.full_like(fresh, c["pages"])), torch.ones_like(fresh, dtype=torch.int32))
    refs += more[:-1]
    lens[dst] = lens[src]
    # reserve: every sequence's growth, in order, from the lowest free pages
    size, grow = lens.long(), s["grow"].long()
    count, after = (size + P - 1) // P, (size + grow + P - 1) // P
    need = after - count
    begin = torch.cumsum(need, 0) - need
    most = c["forks"] * -(-c["grow"] // P)
    fresh = _lowest_free(refs, most)
    here = (col >= count[:, None]) & (col < after[:, None])
    rank = (begin[:, None] + col - count[:, None]).clamp(0, most - 1)
    table.copy_(torch.where(here, fresh[rank].to(torch.int32), table))
    used = torch.arange(most, device=refs.device) < need.sum()
    refs.index_add_(0, fresh, used.to(torch.int32))
    lens += s["grow"]
    # free: the forks' pages given back
    count = (lens[dst].long() + P - 1) // P
    gone = torch.where(col < count[:, None], table[dst], torch.full_like(table[dst], c["pages"])).long().reshape(-1)
    less = torch.zeros(c["pages"] + 1, dtype=torch.int32, device=refs.device)
    less.index_add_(0, gone, torch.ones_like(gone, dtype=torch.int32))
    refs -= less[:-1]
    lens[dst] = 0
    return {"table": table, "lens": lens, "refs": refs, "codes": codes, "scales": scales}


def _plain_compact(s):
    c = s["c"]
    refs, n = s["refs"], c["pages"]
    i = torch.arange(n, device=refs.device)
    live = refs > 0
    total = live.sum()
    free_low, live_high = ~live & (i < total), live & (i >= total)
    slots = torch.zeros(n + 1, dtype=torch.long, device=refs.device)
    spare = torch.full_like(i, n)
    slots[torch.where(free_low, torch.cumsum(free_low, 0) - 1, spare)] = i
    goes = torch.where(live_high, slots[(torch.cumsum(live_high, 0) - 1).clamp(min=0)], i)
    source = torch.arange(n + 1, device=refs.device)
    source[torch.where(live_high, goes, spare)] = i
    source = source[:-1]
    s["codes"].copy_(s["codes"][:, source])
    s["scales"].copy_(s["scales"][:, source])
    col = torch.arange(s["table"].shape[1], device=refs.device)
    count = (s["lens"].long() + c["page"] - 1) // c["page"]
    s["table_out"].copy_(torch.where(col < count[:, None], goes[s["table"].clamp(min=0).long()].to(torch.int32), s["table_out"]))
    s["refs_out"].copy_(torch.where(i < total, refs[source], torch.zeros_like(refs)))
    return {"table": s["table_out"], "refs": s["refs_out"], "codes": s["codes"], "scales": s["scales"]}


_PLAIN = {"w4": _plain_w4, "attend": _plain_attend, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact}


# ------------------------------------------------------------------ the library's calls

def _own_w4(s):
    return _clef.w4_linear(s["x"], s["qw"], s["sw"], s["bias"])


def _own_attend(s):
    return _clef.kv_attention(s["q"], s["codes"], s["scales"], s["table"], s["lens"], causal=s["c"]["causal"])


def _own_append(s):
    _clef.kv_append(s["k"], s["v"], s["codes"], s["scales"], s["table"], s["lens"])
    k, v = _clef.kv_gather(s["codes"], s["scales"], s["table"], s["seq"], s["pos"])
    return {"k": k, "v": v, "scales": s["scales"]}


def _own_fork(s):
    _clef.kv_fork(s["codes"], s["scales"], s["table"], s["lens"], s["refs"], s["src"], s["dst"])
    _clef.kv_reserve(s["table"], s["lens"], s["refs"], s["grow"], s["c"]["page"])
    _clef.kv_free(s["table"], s["lens"], s["refs"], s["dst"], s["c"]["page"])
    return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "codes": s["codes"], "scales": s["scales"]}


def _own_compact(s):
    _clef.kv_compact(s["codes"], s["scales"], s["table"], s["lens"], s["refs"], s["table_out"], s["refs_out"])
    return {"table": s["table_out"], "refs": s["refs_out"], "codes": s["codes"], "scales": s["scales"]}


_OWN = {"w4": _own_w4, "attend": _own_attend, "append": _own_append, "fork": _own_fork, "compact": _own_compact}
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

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "w4":
        # every code by its place in the packed row, spelled out from the layout
        k = torch.arange(c["k"], device="cuda")
        block, j, t, o = k // 128, k % 128 // 32, k % 32 // 8, k % 8
        nibble = o // 2 + 4 * (o % 2)
        byte = block * 64 + t * 16 + j * 4 + nibble // 2
        y = torch.zeros((c["m"], c["n"]), dtype=torch.float64, device="cuda")
        x = s["x"].double()
        for n0 in range(0, c["n"], 4096):
            raw = s["qw"][n0:n0 + 4096][:, byte].to(torch.int16)
            w = ((raw >> (4 * (nibble % 2)).to(torch.int16)) % 16 - 8).double() * s["sw"][n0:n0 + 4096].double()[:, k // c["group"]]
            y[:, n0:n0 + 4096] = torch.einsum("mk,nk->mn", x, w)
        return y if s["bias"] is None else y + s["bias"].double()
    if c["op"] == "attend":
        n, d, P, g = c["n"], c["d"], c["page"], c["hq"] // c["hkv"]
        out = torch.zeros((c["b"] * n, c["hq"], d), dtype=torch.float64, device="cuda")
        for i, size in enumerate(s["lens"].tolist()):
            at = s["table"][i, : -(-size // P)].long()
            for h in range(c["hkv"]):
                raw = s["codes"][:, at, h]
                val = raw.double() if c["kind"] == "int8" else raw.view(torch.float8_e4m3fn).double()
                key, val = (val * s["scales"][:, at, h].double()[..., None, None]).reshape(2, -1, d)[:, :size]
                q = s["q"][i * n:(i + 1) * n, h * g:(h + 1) * g].double().reshape(n * g, d)
                a = torch.einsum("rd,jd->rj", q, key) * d ** -0.5
                if c["causal"]:
                    hidden = torch.ones((n, size), dtype=torch.bool, device="cuda").triu(size - n + 1)
                    a[hidden.repeat_interleave(g, 0)] = float("-inf")
                p = torch.softmax(a, -1).nan_to_num(0.0)
                out[i * n:(i + 1) * n, h * g:(h + 1) * g] = torch.einsum("rj,jd->rd", p, val).view(n, g, d)
        return out
    if c["op"] == "append":
        # page by page: the new scale, the earlier tokens in it, then the new ones
        n, P, top, kind = c["n"], c["page"], _top(c["kind"]), c["kind"]

        def code(v):
            v = v.clamp(-top, top)
            return v.round() if kind == "int8" else v.float().to(torch.float8_e4m3fn).double()

        scales = s["scales"].double()
        new = torch.stack([s["k"], s["v"]]).double()                          # [2][t][h][d]
        rows = []
        for i, size in enumerate(s["lens"].tolist()):
            p = size - n
            while p < size:
                end, held = min(size, (p // P + 1) * P), p % P
                fresh = new[:, i * n + p - (size - n):i * n + end - (size - n)]
                at = int(s["table"][i, p // P])
                was = scales[:, at].clone()
                now = fresh.abs().amax(dim=(1, 3)) / top
                now = torch.maximum(was, now) if held else now
                scales[:, at] = now
                unit = torch.where(now > 0, now, torch.ones_like(now))[:, :, None, None]
                if held:
                    raw = s["codes"][:, at, :, :held]
                    raw = raw.double() if kind == "int8" else raw.view(torch.float8_e4m3fn).double()
                    raw = torch.where((now > was)[:, :, None, None], code(raw * was[:, :, None, None] / unit), raw)
                    rows.append((raw * now[:, :, None, None]).transpose(1, 2))
                q = code(fresh.transpose(1, 2) / unit)
                rows.append((q * now[:, :, None, None]).transpose(1, 2))
                p = end
        k, v = torch.cat(rows, 1).unbind(0)
        return {"k": k, "v": v, "scales": scales}
    return None
