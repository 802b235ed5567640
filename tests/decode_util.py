"""Plain models of the token-by-token operators for the tests, on the CPU: the
packed 4-bit layout, the paged cache's scale rule in IEEE fp32, softmax
attention in fp64 with its error bound, and the page bookkeeping one sequence
at a time."""
from __future__ import annotations

import numpy as np
import torch

TOP = {"int8": 127.0, "e4m3": 448.0}
FLT_MAX = np.float32(3.4028234663852886e38)


# ------------------------------------------------------------------ codes

def encode(v: np.ndarray, kind: str) -> np.ndarray:
    """fp32 -> code bytes (uint8): int8 to nearest even in -127..127, or e4m3 saturating."""
    v = v.astype(np.float32)
    if kind == "int8":
        return np.clip(np.rint(v), -127, 127).astype(np.int8).view(np.uint8)
    return torch.from_numpy(np.clip(v, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def decode(c: np.ndarray, kind: str) -> np.ndarray:
    if kind == "int8":
        return c.view(np.int8).astype(np.float32)
    return torch.from_numpy(np.ascontiguousarray(c)).view(torch.float8_e4m3fn).to(torch.float32).numpy()


def bf16(a) -> np.ndarray:
    """Rounded to bf16, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).to(torch.float32).numpy()


def dev_bf16(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).cuda()


def dev_i32(a) -> torch.Tensor:
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def dev_codes(c: np.ndarray, kind: str) -> torch.Tensor:
    t = torch.from_numpy(c.copy()).cuda()
    return t.view(torch.int8) if kind == "int8" else t


def host_codes(t: torch.Tensor) -> np.ndarray:
    return t.detach().contiguous().view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------ 4-bit rows

def w4_places(K: int):
    """(byte, shift) of each weight of a packed row."""
    k = np.arange(K)
    block, j, t, o = k // 128, k % 128 // 32, k % 32 // 8, k % 8
    nibble = o // 2 + 4 * (o % 2)
    return block * 64 + 16 * t + 4 * j + nibble // 2, 4 * (nibble % 2)


def w4_codes(qw: np.ndarray, K: int) -> np.ndarray:
    byte, shift = w4_places(K)
    return ((qw[:, byte].astype(np.int64) >> shift) & 15) - 8


def w4_pack(codes: np.ndarray) -> np.ndarray:
    N, K = codes.shape
    kp = (K + 127) // 128 * 128
    full = np.zeros((N, kp), np.int64)
    full[:, :K] = codes
    byte, shift = w4_places(kp)
    out = np.zeros((N, kp // 2), np.int64)
    np.add.at(out, (slice(None), byte), (full + 8) << shift)
    return out.astype(np.uint8)


# ------------------------------------------------------------------ cache

class Cache:
    """A pool with the rule of the cache's append in IEEE fp32."""

    def __init__(self, kind, pages, heads, page, dim, planes=2, seed=0, fill=0xFF):
        self.kind, self.P, self.D = kind, page, dim
        # what no token has been written to: NaN codes (e4m3) and scales that would show
        self.codes = np.full((planes, pages, heads, page, dim), fill, np.uint8)
        self.scales = np.full((planes, pages, heads), 1e30, np.float32)

    def append(self, row, length, new):
        """new: fp32 [2][n][heads][dim], the last n of `length` tokens."""
        n, P, top = new.shape[1], self.P, np.float32(TOP[self.kind])
        p = length - n
        while p < length:
            end, held, at = min(length, (p // P + 1) * P), p % P, row[p // P]
            part = new[:, p - (length - n):end - (length - n)]
            amax = np.abs(part).max(axis=(1, 3)).astype(np.float32)
            old = self.scales[:, at].copy() if held else np.zeros_like(amax)
            s = np.maximum(old, amax / top)
            with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
                r = np.where(s > 0, np.minimum(np.float32(1) / s, FLT_MAX), np.float32(0)).astype(np.float32)
                f = np.where(s > 0, old / s, np.float32(1)).astype(np.float32)
            for pl, h in np.ndindex(*s.shape):
                if held and s[pl, h] > old[pl, h]:
                    was = decode(self.codes[pl, at, h, :held], self.kind)
                    self.codes[pl, at, h, :held] = encode(was * f[pl, h], self.kind)
                self.codes[pl, at, h, held:held + end - p] = encode(part[pl, :, h] * r[pl, h], self.kind)
            self.scales[:, at] = s
            p = end

    def values(self, row, length):
        """fp64 [2][length][heads][dim]."""
        at = np.asarray(row[: -(-length // self.P)], np.int64)
        v = decode(self.codes[:, at], self.kind).astype(np.float64) * self.scales[:, at].astype(np.float64)[..., None, None]
        pl, n, h, P, d = v.shape
        return v.transpose(0, 1, 3, 2, 4).reshape(pl, n * P, h, d)[:, :length]

    def device(self):
        return dev_codes(self.codes, self.kind), torch.from_numpy(self.scales.copy()).cuda()


def scattered_table(rng, lens, page, spare=2, width=None):
    """A page table of shuffled pages for the lengths: (table, pages)."""
    counts = [-(-x // page) for x in lens]
    pages = sum(counts) + spare
    perm = rng.permutation(pages)
    width = width or max(counts + [1])
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for i, c in enumerate(counts):
        table[i, :c] = perm[at:at + c]
        at += c
    return table, pages


def filled_cache(rng, kind, lens, heads, page, dim, spread=2.0):
    """A cache whose sequences hold random tokens, with tables and lengths."""
    table, pages = scattered_table(rng, lens, page)
    c = Cache(kind, pages, heads, page, dim)
    for i, x in enumerate(lens):
        if x:
            new = bf16(rng.standard_normal((2, x, heads, dim)) * np.exp(spread * rng.standard_normal((2, x, heads, 1)) * 0.3))
            c.append(table[i], x, new)
    return c, table, pages


# ------------------------------------------------------------------ attention

def attention(q, kv, scale, causal):
    """One sequence in fp64: q [n][hq][d], kv [2][len][h][d].  Returns (out, lse,
    bound of the kernel's error of out before its bf16 rounding, bound of lse).

    The bound: x = scale q.k is off by at most dx (fp32 sums of d products in
    16-deep steps, the queries' fp16 form, a few fp32 roundings), so a weight
    is off by exp(2 dx) - 1 with the sum's own error, by 2^-11 for its rounding
    to fp16 and 2^-18 for the exponentials and the fp32 sums; weights times
    scale under 2^-14 of the largest are off by 2^-25 of it each."""
    n, hq, d = q.shape
    L, h = kv.shape[1], kv.shape[2]
    g = hq // h
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    tol, tol_lse = np.zeros((n, hq, d)), np.zeros((n, hq))
    for i in range(n):
        end = min(L, max(0, L - n + i + 1)) if causal else L
        if end == 0:
            continue
        for j in range(hq):
            k, v = kv[0, :end, j // g], kv[1, :end, j // g]
            x = scale * (k @ q[i, j])
            m = x.max()
            w = np.exp(x - m)
            p = w / w.sum()
            out[i, j] = p @ v
            lse[i, j] = m + np.log(w.sum())
            mag = np.abs(k) @ np.abs(q[i, j])
            dx = abs(scale) * ((d / 16 + 4) * 2.0 ** -23 * mag.max() + 2.0 ** -37 * np.abs(q[i, j]).max() * np.abs(k).sum(1).max())
            dx += 2.0 ** -21 * np.abs(x).max()
            rel = np.expm1(2 * dx) + 2.0 ** -11 + 2.0 ** -18
            tol[i, j] = rel * (p @ np.abs(v)) + end * 2.0 ** -24 * (p[:, None] * np.abs(v)).max()
            tol_lse[i, j] = dx + 2.0 ** -18 + 2.0 ** -22 * abs(lse[i, j])
    return out, lse, tol, tol_lse


def bf16_ulp(v):
    a = np.maximum(np.abs(np.asarray(v, np.float64)), 2.0 ** -126)
    return 2.0 ** (np.floor(np.log2(a)) - 7)


# ------------------------------------------------------------------ pages

class Pages:
    """The bookkeeping one sequence at a time."""

    def __init__(self, table, lens, refs, page):
        self.table, self.lens, self.refs, self.P = table.copy(), list(lens), refs.copy(), page

    def _lowest(self):
        free = np.flatnonzero(self.refs == 0)
        return int(free[0])

    def reserve(self, grow):
        need = sum(-(-(x + g) // self.P) - -(-x // self.P) for x, g in zip(self.lens, grow))
        if need > (self.refs == 0).sum():
            return False
        for b, g in enumerate(grow):
            for i in range(-(-self.lens[b] // self.P), -(-(self.lens[b] + g) // self.P)):
                p = self._lowest()
                self.refs[p] = 1
                self.table[b, i] = p
            self.lens[b] += g
        return True

    def fork(self, src, dst):
        """Returns the page copies, or None if there are too few free pages."""
        if sum(self.lens[s] % self.P != 0 for s in src) > (self.refs == 0).sum():
            return None
        moves = []
        for s, d in zip(src, dst):
            full = self.lens[s] // self.P
            if self.lens[s] % self.P:
                p = self._lowest()
                self.refs[p] = 1
                moves.append((int(self.table[s, full]), p))
                self.table[d, full] = p
        for s, d in zip(src, dst):
            full = self.lens[s] // self.P
            self.table[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                self.refs[p] += 1
            self.lens[d] = self.lens[s]
        return moves

    def free(self, seqs):
        for b in seqs:
            for p in self.table[b, : -(-self.lens[b] // self.P)]:
                self.refs[p] -= 1
            self.lens[b] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        gaps = [p for p in range(live) if self.refs[p] == 0]
        high = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        goes = dict(zip(high, gaps))
        for b, x in enumerate(self.lens):
            for i in range(-(-x // self.P)):
                self.table[b, i] = goes.get(int(self.table[b, i]), self.table[b, i])
        for a, z in goes.items():
            self.refs[z], self.refs[a] = self.refs[a], 0
        return live, list(goes.items())
