"""GPU: examples/paged_decode.py (4-bit weights, append, prefill, decode, fork,
window, free, compact together) against dense attention in binary64 over the
tokens that each sequence has seen."""
import os
import sys

import numpy as np
import pytest
import torch

import kv_ref as R
from gpu_util import say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import paged_decode as E  # noqa: E402

pytestmark = pytest.mark.gpu


class Dense:
    """The same layers with weights in full and every token kept."""

    def __init__(self, fmt, seed):
        import bit_block_quantized_nibble_amd as qbn

        d = E.Decoder(fmt, 6, 32, 96, seed=seed)
        full = lambda w: qbn.dequantize(w).double().cpu().numpy()  # noqa: E731
        self.qkv, self.out, self.fmt = [full(w) for w in d.qkv], [full(w) for w in d.out], fmt
        self.kept = {}  # slot -> per layer (K rows, V rows)

    def held(self, x):
        """What the cache holds of x [tokens][KV][DIM]."""
        x = torch.from_numpy(x).bfloat16().double().numpy()
        if self.fmt == "bf16":
            return x
        code, scale = R.quantize(self.fmt, x)
        grid = R.FP4 if self.fmt == "mxfp4" else R.FP8
        return grid[code] * np.repeat(R.e8m0(scale), 32, -1)

    def forward(self, slot, x):
        kept = self.kept.setdefault(slot, [([], []) for _ in range(E.LAYERS)])
        for i in range(E.LAYERS):
            v = torch.from_numpy(x @ self.qkv[i].T).bfloat16().double().numpy().reshape(len(x), -1, E.DIM)
            k, w = self.held(v[:, E.HEADS:E.HEADS + E.KV]), self.held(v[:, E.HEADS + E.KV:])
            kept[i][0].extend(k), kept[i][1].extend(w)
            K, V = np.stack(kept[i][0]), np.stack(kept[i][1])
            o = np.zeros((len(x), E.HEADS, E.DIM))
            for t in range(len(x)):
                for h in range(E.HEADS):
                    kv = h // (E.HEADS // E.KV)
                    o[t, h] = R.attention(v[t, h], K[:, kv], V[:, kv], len(K) - len(x) + t, E.WINDOW, E.SINKS, E.DIM ** -0.5)[0]
            o = torch.from_numpy(o).bfloat16().double().numpy().reshape(len(x), -1)
            y = torch.from_numpy(o @ self.out[i].T).bfloat16().double().numpy()
            x = torch.from_numpy(x + y).bfloat16().double().numpy()
        return x


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
def test_example_matches_dense_attention(fmt):
    prompts = (37, 130, 64)
    ref = Dense(fmt, 0)
    seen = []
    for what, slots, x, y, word in E.serve(fmt, 12, prompts):
        say(fmt, what, slots)
        seen.append(what)
        if what == "fork":
            assert int(word) == -1
            ref.kept[3] = [(list(k), list(v)) for k, v in ref.kept[0]]
            continue
        if what == "leave":
            assert 0 < int(word) < 96
            continue
        assert int(word) == -1
        x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
        at = 0
        for i, s in enumerate(slots):
            n = prompts[i] if what == "prefill" else 1
            want = ref.forward(s, x[at:at + n])
            # every stage rounds to bfloat16 (2^-8 of values near 1, twice a
            # layer), and a rounding of K or V that falls the other way moves
            # an MX element by a step: held to the root mean square
            err = np.sqrt(np.mean((y[at:at + n] - want) ** 2) / np.mean(want ** 2))
            assert err < (2.0 ** -7 if fmt == "bf16" else 2.0 ** -5), "%s slot %d: relative error %g" % (what, s, err)
            at += n
    assert seen.count("step") == 12 and "fork" in seen and "leave" in seen
