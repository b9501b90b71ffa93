"""A small decoder's attention layers with 4-bit weights and a paged cache, served.

Three prompts of different lengths are prefilled, every sequence then takes
one token a step. Between steps the first sequence forks (its beam goes on from
the shared pages), the second one leaves, what slid out of the window is given
back and the pool is packed. Weights are MXFP4 (quantized_gemm), the cache is
bfloat16, MXFP8 or MXFP4.

    python examples/paged_decode.py [--format mxfp4] [--steps 24]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_block_quantized_nibble_amd as qbn  # noqa: E402

HIDDEN, HEADS, KV, DIM, PAGE, LAYERS = 512, 8, 2, 64, 16, 2
WINDOW, SINKS = 96, 4


def ints(v, device):
    return torch.tensor(v, dtype=torch.int32, device=device)


def weight(n: int, k: int, g: torch.Generator, device) -> qbn.QTensor:
    codes, scales = qbn.quantize_mx(torch.randn(n, k, generator=g, device=device) * k ** -0.5)
    return qbn.QTensor("mxfp4", n, k, codes, scales)


class Decoder:
    """Layers of x + Wo attention(Wqkv x) over one paged cache."""

    def __init__(self, fmt: str, slots: int, row: int, pages: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.wide = HEADS + 2 * KV
        self.qkv = [weight(self.wide * DIM, HIDDEN, g, device) for _ in range(LAYERS)]
        self.out = [weight(HIDDEN, HEADS * DIM, g, device) for _ in range(LAYERS)]
        self.cache = qbn.KVCache.empty(fmt, LAYERS, pages, KV, PAGE, DIM, device=device)
        self.pool = qbn.KVPool.empty(slots, row, pages, PAGE, device=device)
        self.device = device

    def forward(self, x: torch.Tensor, rows: torch.Tensor, cu) -> torch.Tensor:
        """x [tokens][HIDDEN] of the sequences in slots `rows`, whose room is
        reserved; cu: int32 [len(rows) + 1], or None for one token each."""
        table, lens = self.pool.table[rows.long()], self.pool.lens[rows.long()]
        for i in range(LAYERS):
            v = qbn.quantized_gemm(self.qkv[i], x).view(-1, self.wide, DIM)
            qbn.kv_append(self.cache, v[:, HEADS:HEADS + KV], v[:, HEADS + KV:], table, lens, cu, layer=i)
            if cu is None:
                a, _ = qbn.kv_attention_decode(self.cache, v[:, :HEADS], table, lens, WINDOW, SINKS, layer=i)
            else:
                a, _ = qbn.kv_attention_prefill(self.cache, v[:, :HEADS], cu, table, lens, WINDOW, SINKS, layer=i)
            x = x + qbn.quantized_gemm(self.out[i], a.view(-1, HEADS * DIM))
        return x


def serve(fmt: str = "mxfp4", steps: int = 24, prompts=(37, 130, 64), device="cuda", seed: int = 0):
    """Yields (what, slots, x in, x out, pages in use) after each forward pass."""
    d = Decoder(fmt, slots=6, row=32, pages=96, device=device, seed=seed)
    g = torch.Generator(device=device)
    g.manual_seed(seed + 1)
    tokens = lambda n: torch.randn(n, HIDDEN, generator=g, device=device).bfloat16()  # noqa: E731

    slots = list(range(len(prompts)))
    ok = qbn.kv_reserve(d.pool, ints(slots, device), ints(prompts, device))
    cu = [0]
    for n in prompts:
        cu.append(cu[-1] + n)
    x = tokens(cu[-1])
    y = d.forward(x, ints(slots, device), ints(cu, device))
    yield "prefill", list(slots), x, y, ok
    for step in range(steps):
        if step == steps // 3:  # a second beam of the first sequence
            ok = qbn.kv_fork(d.cache, d.pool, ints([0], device), ints([3], device))
            slots.append(3)
            yield "fork", [0, 3], None, None, ok
        if step == 2 * steps // 3:  # the second sequence is done; old pages go, the rest is packed
            slots.remove(1)
            qbn.kv_free(d.pool, ints([1], device))
            qbn.kv_free(d.pool, ints(slots, device), window=WINDOW, sinks=SINKS)
            live = qbn.kv_compact(d.cache, d.pool)
            yield "leave", [1], None, None, live
        rows = ints(slots, device)
        ok = qbn.kv_reserve(d.pool, rows, ints([1] * len(slots), device))
        x = tokens(len(slots))
        y = d.forward(x, rows, None)
        yield "step", list(slots), x, y, ok


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--format", default="mxfp4", choices=("bf16", "mxfp8", "mxfp4"))
    p.add_argument("--steps", type=int, default=24)
    a = p.parse_args()
    for what, slots, _, y, word in serve(a.format, a.steps):
        if what == "leave":
            print("sequence 1 leaves; %d pages in use" % int(word))
        elif int(word) != -1:
            raise SystemExit("%s: request %d could not be met" % (what, int(word)))
        elif what == "fork":
            print("sequence 0 forks into slot 3")
        else:
            print("%-7s slots %s: mean square of the outputs %.4f" % (what, slots, float(y.float().square().mean())))


if __name__ == "__main__":
    main()
