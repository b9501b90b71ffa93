"""A small decoder with rotary positions, a paged cache and experts in 4 bits, served.

Each layer is x + Wo attention(Wqkv x), with queries and keys turned by their
positions on the way into the cache (kv_append_rope), and x + experts(x), a few of
many for each token (moe). Prompts of different lengths are prefilled, then every
sequence takes one token a step. Weights of the projections are MXFP4, the
experts' MXFP4 or NVFP4, the cache is bfloat16, MXFP8 or MXFP4.

    python examples/moe_decode.py [--format mxfp4] [--experts nvfp4] [--steps 16]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_block_quantized_nibble_amd as qbn  # noqa: E402

HIDDEN, HEADS, KV, DIM, ROT, PAGE, LAYERS = 512, 8, 2, 64, 32, 16, 2
EXPERTS, TOP, INTER = 16, 4, 256


def ints(v, device):
    return torch.tensor(v, dtype=torch.int32, device=device)


def matrix(n: int, k: int, g: torch.Generator, device) -> torch.Tensor:
    return torch.randn(n, k, generator=g, device=device) * k ** -0.5


def projection(n: int, k: int, g: torch.Generator, device) -> qbn.QTensor:
    return qbn.QTensor("mxfp4", n, k, *qbn.quantize_mx(matrix(n, k, g, device)))


def experts(fmt: str, g: torch.Generator, device) -> qbn.MoE:
    """Experts quantized one matrix at a time, stacked, with a router over them."""
    parts = []
    for n, k in ((2 * INTER, HIDDEN), (HIDDEN, INTER)):
        ws = [matrix(n, k, g, device) for _ in range(EXPERTS)]
        if fmt == "mxfp4":
            made, factor = [qbn.quantize_mx(w) for w in ws], None
        else:  # a factor per expert, so that the largest block's scale is E4M3's largest, 448
            tops = [float(w.abs().max()) / (6.0 * 448.0) for w in ws]
            made, factor = [qbn.quantize_nvfp4(w, t) for w, t in zip(ws, tops)], torch.tensor(tops, device=device)
        parts += [torch.stack([c for c, _ in made]), torch.stack([s for _, s in made]), factor]
    router = qbn.MoERouter((matrix(EXPERTS, HIDDEN, g, device) * 2).bfloat16(), TOP)
    return qbn.MoE(fmt, router, parts[0], parts[1], parts[3], parts[4], w13_scale2=parts[2], w2_scale2=parts[5])


class Decoder:
    def __init__(self, fmt: str, experts_fmt: str, slots: int, row: int, pages: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.wide = HEADS + 2 * KV
        self.qkv = [projection(self.wide * DIM, HIDDEN, g, device) for _ in range(LAYERS)]
        self.out = [projection(HIDDEN, HEADS * DIM, g, device) for _ in range(LAYERS)]
        self.moe = [experts(experts_fmt, g, device) for _ in range(LAYERS)]
        self.rope = qbn.Rope.make(ROT, scaling="yarn", scale=4.0, original=256, device=device)
        self.cache = qbn.KVCache.empty(fmt, LAYERS, pages, KV, PAGE, DIM, device=device)
        self.pool = qbn.KVPool.empty(slots, row, pages, PAGE, device=device)

    def forward(self, x: torch.Tensor, rows: torch.Tensor, cu, watch=None) -> torch.Tensor:
        """x [tokens][HIDDEN] of the sequences in slots `rows`, whose room is
        reserved; cu: int32 [len(rows) + 1], or None for one token each. watch:
        called with every stage's name, layer and tensors."""
        watch = watch or (lambda *a: None)
        table, lens = self.pool.table[rows.long()], self.pool.lens[rows.long()]
        for i in range(LAYERS):
            v = qbn.quantized_gemm(self.qkv[i], x).view(-1, self.wide, DIM)
            q, k, w = v.split((HEADS, KV, KV), 1)
            turned = qbn.kv_append_rope(self.cache, q, k, w, table, lens, self.rope, cu, layer=i)
            if cu is None:
                a, _ = qbn.kv_attention_decode(self.cache, turned, table, lens, layer=i)
            else:
                a, _ = qbn.kv_attention_prefill(self.cache, turned, cu, table, lens, layer=i)
            watch("attention", i, v, turned, a)
            x = x + qbn.quantized_gemm(self.out[i], a.view(-1, HEADS * DIM))
            y, ids, weights = qbn.moe(self.moe[i], x)
            watch("experts", i, x, y, ids, weights)
            x = x + y
        return x


def serve(fmt: str = "mxfp4", experts_fmt: str = "mxfp4", steps: int = 16, prompts=(37, 5, 64), device="cuda", seed: int = 0,
          watch=None):
    """Yields (what, decoder, x in, x out, status) after each forward pass."""
    d = Decoder(fmt, experts_fmt, slots=len(prompts), row=16, pages=64, device=device, seed=seed)
    g = torch.Generator(device=device)
    g.manual_seed(seed + 1)
    tokens = lambda n: torch.randn(n, HIDDEN, generator=g, device=device).bfloat16()  # noqa: E731
    rows = ints(range(len(prompts)), device)
    cu = [0]
    for n in prompts:
        cu.append(cu[-1] + n)
    ok = qbn.kv_reserve(d.pool, rows, ints(prompts, device))
    x = tokens(cu[-1])
    yield "prefill", d, x, d.forward(x, rows, ints(cu, device), watch), ok
    for _ in range(steps):
        ok = qbn.kv_reserve(d.pool, rows, ints([1] * len(prompts), device))
        x = tokens(len(prompts))
        yield "step", d, x, d.forward(x, rows, None, watch), ok


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--format", default="mxfp4", choices=("bf16", "mxfp8", "mxfp4"))
    p.add_argument("--experts", default="mxfp4", choices=("mxfp4", "nvfp4"))
    p.add_argument("--steps", type=int, default=16)
    a = p.parse_args()
    for what, _, _, y, ok in serve(a.format, a.experts, a.steps):
        if int(ok) != -1:
            raise SystemExit("%s: request %d could not be met" % (what, int(ok)))
        print("%-7s %d tokens: mean square of the outputs %.4f" % (what, len(y), float(y.float().square().mean())))


if __name__ == "__main__":
    main()
