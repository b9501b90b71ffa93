"""GPU: silu of gates far from zero, where its exponential passes binary32's range."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
from gpu_util import DEV, say
from test_gpu_moe import make, to
from test_gpu_moe_halves import one_hot

pytestmark = pytest.mark.gpu

GATES = [0.0, -0.0, 1e-30, -1e-30, 2.0, -2.0, 17.0, -17.0, -60.0, 80.0, -80.0, -87.0, -87.5, -88.0, -89.0, 89.0, -96.0, -104.0,
         -128.0, 128.0, -1e4, 1e4, -1e20, 1e20, -3e38, 3e38]


@pytest.mark.parametrize("tokens", [8, len(GATES)])
@pytest.mark.parametrize("up", [2.0 ** -20, 1.0, 2.0 ** 40])
def test_gates_far_from_zero(tokens, up):
    """h = silu(gate) * up, the output. silu is off by 2^-119 where its exponential passes
    2^126; else by the exponent's rounding (2 |gate| U of it) and 4 U, U = 2^-24."""
    rows = [(0, 0, 1), (32, 1, 1)]
    one = np.full((1, 64, 1), 127, np.uint8)
    layer = make([one_hot(64, 32, rows)[None], one, None, one_hot(32, 32, [(0, 0, 1)])[None], one[:, :32].copy(), None], "mxfp4")
    for first in range(0, len(GATES), tokens):
        gates = (GATES[first:] + GATES)[:tokens]
        x = torch.zeros(tokens, 32, dtype=torch.float64)
        x[:, 0], x[:, 1] = torch.tensor(gates, dtype=torch.float64), up
        x = x.bfloat16()
        say("gates", tokens, up, first)
        got = qbn.moe_experts(layer, x.to(DEV), to(np.zeros((tokens, 1), np.int32)), to(np.ones((tokens, 1), np.float32)))
        g = x[:, 0].double().numpy()
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        off = np.where(g < -87, 2.0 ** -119, 0) + np.abs(silu) * (2 * np.abs(g) * (g < 0) + 4) * 2.0 ** -24
        with np.errstate(over="ignore"):
            want, tol = silu * up, off * up + np.abs(silu * up) * 2.0 ** -16
        got, most = got[:, 0].cpu().double().numpy(), float(torch.finfo(torch.bfloat16).max)
        fits = np.abs(want) < most
        assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134)[fits].all(), (got, want)
        assert np.isposinf(got[~fits]).all()
