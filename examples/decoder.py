"""Example: a stack of decoder layers that reads prompts and answers token by token.

``Decoder`` holds each projection twice: as INT8 codes for the W8A8 GEMMs that
read prompts (many rows: tensor-bound) and as 4-bit codes for the linears that
answer (a row or a few: bound by the bytes of the weights).  All sequences
share one pool of 8-bit key and value pages; a prompt that is answered several
ways is read once and forked, its pages shared.  Everything that a step needs
-- lengths, page tables, counts -- stays on the device, so a step launches
kernels only and can be captured in a CUDA graph (``capture``), which also
takes the host's cost per call out of short steps.

RMS normalisation, the rotation of queries and keys by their position and the
residual adds are torch's elementwise operations here; they are not part of the library.

    PYTHONPATH=. python examples/decoder.py        # random weights: a prompt, three answers of 40 tokens
"""
from __future__ import annotations

from typing import Dict, List, Sequence

import torch

from w8a8_quantized_projections_gb300 import (kv_append, kv_attention, kv_compact, kv_fork, kv_free, kv_reserve, poll_status,
                                              quant_act, quant_w4, swiglu_bf16, w4_linear, w8a8_gateup_swiglu, w8a8_linear)

NAMES = ("qkv", "o", "gateup", "down")


class Decoder:
    def __init__(self, layers: List[Dict[str, torch.Tensor]], q_heads: int, kv_heads: int, dim: int, sequences: int,
                 pages: int, width: int, page: int = 64, kind: str = "int8", group: int = 128, theta: float = 10000.0,
                 eps: float = 1e-6):
        """layers: for each layer bf16 weights "qkv" [(q_heads + 2 kv_heads) dim][hidden],
        "o" [hidden][q_heads dim], "gateup" [2 F][hidden], "down" [hidden][F] and the
        norms' "norm_attn" and "norm_mlp" [hidden];
        sequences: how many there can be; pages: pages of the pool, each `page`
        tokens of every layer; width: pages a sequence can have;
        kind: "int8" or "e4m3" cache codes; group: weights that share a scale."""
        if kind not in ("int8", "e4m3"):
            raise ValueError(f"kind {kind!r}: int8 or e4m3")
        device = layers[0]["qkv"].device
        self.q_heads, self.kv_heads, self.dim, self.page, self.eps = q_heads, kv_heads, dim, page, eps
        self.norms = [(w["norm_attn"].float(), w["norm_mlp"].float()) for w in layers]
        self.w8 = [{n: quant_act(w[n], "int8_h128") for n in NAMES} for w in layers]
        self.w4 = [{n: quant_w4(w[n], group) for n in NAMES} for w in layers]
        code = torch.int8 if kind == "int8" else torch.float8_e4m3fn
        self.codes = torch.zeros((2 * len(layers), pages, kv_heads, page, dim), dtype=torch.uint8, device=device).view(code)
        self.scales = torch.zeros((2 * len(layers), pages, kv_heads), dtype=torch.float32, device=device)
        self.table = torch.zeros((sequences, width), dtype=torch.int32, device=device)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.rows = torch.zeros(sequences + 1, dtype=torch.int32, device=device)      # of a reservation
        self.numbers = torch.arange(sequences + 1, dtype=torch.int32, device=device)
        self.freq = theta ** (-torch.arange(0, dim, 2, dtype=torch.float32, device=device) / dim)
        self.graph = None

    # ------------------------------------------------------------ running

    def prompt(self, x: torch.Tensor, counts: Dict[int, int]) -> torch.Tensor:
        """Reads x (bf16 [rows][hidden]) on the ends of sequences: counts[s] rows for
        sequence s, in the order of `counts`.  Returns the rows' hidden states."""
        if sum(counts.values()) != x.shape[0] or min(counts.values(), default=0) < 0:
            raise ValueError(f"counts of {sum(counts.values())} rows for {x.shape[0]}")
        seqs = self._ids(list(counts))
        n = torch.tensor(list(counts.values()), dtype=torch.int32, device=x.device)
        start = torch.zeros(len(counts) + 1, dtype=torch.int32, device=x.device)
        torch.cumsum(n, 0, dtype=torch.int32, out=start[1:])
        table, lens, rows = self._grow(seqs, n)
        seq_of = torch.repeat_interleave(torch.arange(len(counts), device=x.device), n.long(), output_size=x.shape[0])
        # row r is token len - n + (r - start) of its sequence
        at = torch.arange(x.shape[0], device=x.device) + (lens - start[1:])[seq_of]
        return self._run(x, at, table, lens, torch.minimum(start, rows), start, self._many_rows)

    def step(self, x: torch.Tensor, seqs: Sequence[int] | torch.Tensor) -> torch.Tensor:
        """One token on the end of each sequence listed: x bf16 [len(seqs)][hidden].  Where the pool
        has no page left for one of them, none grows, the cache stays as it is, the result
        means nothing and poll_status() is 6."""
        seqs = self._ids(seqs)
        if x.shape[0] != seqs.shape[0]:
            raise ValueError(f"{x.shape[0]} rows for {seqs.shape[0]} sequences")
        table, lens, rows = self._grow(seqs, torch.ones_like(seqs))
        return self._run(x, lens - 1, table, lens, torch.minimum(self.numbers[: len(seqs) + 1], rows), None, self._few_rows)

    def capture(self, x: torch.Tensor, seqs: Sequence[int]) -> torch.Tensor:
        """Records step(x, seqs) into a CUDA graph and returns the tensor that
        ``replay()`` fills; refill x in place for the next token.  Recording runs
        nothing: the sequences are as before the call."""
        seqs = self._ids(seqs)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        self._captured = (x, seqs)
        with torch.cuda.graph(self.graph):
            self.out = self.step(x, seqs)
        return self.out

    def replay(self) -> torch.Tensor:
        self.graph.replay()
        return self.out

    # ------------------------------------------------------------ sequences

    def fork(self, src: Sequence[int], dst: Sequence[int]) -> None:
        """Each sequence of dst, empty before, goes on from the tokens of the one of src."""
        kv_fork(self.codes, self.scales, self.table, self.lens, self.refs, self._ids(src, False), self._ids(dst))

    def free(self, seqs: Sequence[int]) -> None:
        kv_free(self.table, self.lens, self.refs, self._ids(seqs), self.page)

    def compact(self) -> torch.Tensor:
        """Moves the held pages to the pool's start; their number, on the device."""
        return kv_compact(self.codes, self.scales, self.table, self.lens, self.refs)

    # ------------------------------------------------------------ parts

    def _ids(self, seqs, different=True) -> torch.Tensor:
        if isinstance(seqs, torch.Tensor):
            return seqs
        if not all(0 <= s < self.lens.shape[0] for s in seqs) or different and len(set(seqs)) != len(seqs):
            raise ValueError(f"sequences {list(seqs)}: {'different ones of ' if different else ''}0..{self.lens.shape[0] - 1}")
        return torch.tensor(list(seqs), dtype=torch.int32, device=self.lens.device)

    def _grow(self, seqs, n):
        """The sequences' pages and lengths with n more tokens, and how many rows were given a
        place: all, or none where the pool is full."""
        grow = torch.zeros_like(self.lens).index_copy_(0, seqs.long(), n)
        kv_reserve(self.table, self.lens, self.refs, grow, self.page, row_start=self.rows)
        return self.table.index_select(0, seqs), self.lens.index_select(0, seqs), self.rows[-1:]

    def _run(self, x, at, table, lens, placed, start, project):
        hq, hk, d = self.q_heads, self.kv_heads, self.dim
        angle = at.to(torch.float32)[:, None] * self.freq
        cos, sin = angle.cos()[:, None], angle.sin()[:, None]
        for i, (norm_attn, norm_mlp) in enumerate(self.norms):
            codes, scales = self.codes[2 * i : 2 * i + 2], self.scales[2 * i : 2 * i + 2]
            qkv = project(i, "qkv", self._norm(x, norm_attn)).view(-1, hq + 2 * hk, d)
            qk = self._rotate(qkv[:, : hq + hk], cos, sin)
            kv_append(qk[:, hq:], qkv[:, hq + hk :], codes, scales, table, lens, placed)
            o = kv_attention(qk[:, :hq], codes, scales, table, lens, start)
            x = x + project(i, "o", o.view(-1, hq * d))
            x = x + project(i, "down", project(i, "gateup", self._norm(x, norm_mlp)))
        return x

    def _many_rows(self, i, name, a):
        q, s = quant_act(a, "int8_h128")
        return (w8a8_gateup_swiglu if name == "gateup" else w8a8_linear)(q, s, *self.w8[i][name])

    def _few_rows(self, i, name, a):
        y = w4_linear(a, *self.w4[i][name])
        return swiglu_bf16(y) if name == "gateup" else y

    def _norm(self, x, w):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + self.eps) * w).to(torch.bfloat16)

    @staticmethod
    def _rotate(t, cos, sin):
        a, b = t.float().chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(torch.bfloat16)


def main():
    hidden, q_heads, kv_heads, dim, ff, depth = 2048, 16, 4, 128, 5632, 4

    def w(n, k):
        return (torch.randn(n, k, device="cuda") * k ** -0.5).to(torch.bfloat16)

    one = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    dec = Decoder([{"qkv": w((q_heads + 2 * kv_heads) * dim, hidden), "o": w(hidden, q_heads * dim), "gateup": w(2 * ff, hidden),
                    "down": w(hidden, ff), "norm_attn": one, "norm_mlp": one} for _ in range(depth)],
                  q_heads, kv_heads, dim, sequences=8, pages=256, width=64)
    table = torch.randn(1000, hidden, device="cuda").to(torch.bfloat16)       # tokens' vectors, in and out
    h = dec.prompt(table[torch.randint(1000, (1502,), device="cuda")], {0: 1502})
    dec.fork([0, 0], [1, 2])
    token = (h[-1].float() @ table.float().T).topk(3).indices                  # three first tokens
    x = table[token].clone()
    y = dec.capture(x, [0, 1, 2])

    def tokens(n):
        for _ in range(n):
            dec.replay()
            x.copy_(table[(y.float() @ table.float().T).argmax(-1)])

    tokens(8)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    tokens(32)
    end.record()
    torch.cuda.synchronize()
    status = poll_status()
    print(f"{dec.lens.tolist()[:3]} tokens, {start.elapsed_time(end) / 32 * 1000:.0f} us a token of three answers, status {status}")
    dec.free([1, 2])
    print(f"{int(dec.compact())} pages held after two answers are freed")


if __name__ == "__main__":
    main()
