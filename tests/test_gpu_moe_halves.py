"""GPU: how much of h its two bfloat16 parts keep, seen where the second product takes
nearly all of it off again."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
from gpu_util import DEV, say
from test_gpu_moe import make, to

pytestmark = pytest.mark.gpu


def one_hot(rows, k, at):
    """E2M1 codes [rows][k / 2] that are 1 (or -1) at (row, column, sign)."""
    c = np.zeros((rows, k), np.uint8)
    for r, i, sign in at:
        c[r, i] = 2 if sign > 0 else 10
    return c[:, 0::2] | c[:, 1::2] << 4


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("tokens", [8, 1024])
def test_parts_of_h(fmt, tokens):
    """h_0 = 2^17 + r for every r below 2^10, h_1 = 2^17 + r to the nearest 64 (two
    bfloat16 numbers hold it), out = h_0 - h_1, at most 32 in magnitude: exact but for
    h_0's parts. The first is h_0 rounded to 8 bits, so that at most half of its last
    bit is left, 2^9; that rounded to 8 bits is off by half of its last one, 2^0 at
    most: 2^-17 of h."""
    r = np.arange(1024) if tokens == 1024 else np.array([513, 514, 515, 600, 770, 1021, 1022, 1023])
    m = np.floor(r / 64 + 0.5)
    x = np.zeros((tokens, 32), np.float32)
    # silu(64) is 64 in binary32; the up projections are sums of exact products: h / 64
    x[:, 0], x[:, 1], x[:, 2], x[:, 3], x[:, 4] = 64, 2048, (r & ~127) / 64, (r & 127) / 64, m
    rows = [(0, 0, 1), (1, 0, 1), (32, 1, 1), (32, 2, 1), (32, 3, 1), (33, 1, 1), (33, 4, 1)]
    one = np.full((1, 64, 1), 127, np.uint8) if fmt == "mxfp4" else np.full((1, 64, 2), 0x38, np.uint8)
    f = None if fmt == "mxfp4" else np.ones(1, np.float32)
    parts = [one_hot(64, 32, rows)[None], one, f, one_hot(32, 32, [(0, 0, 1), (0, 1, -1)])[None], one[:, :32].copy(), f]
    x = torch.from_numpy(x)
    assert torch.equal(x.bfloat16().float(), x)
    say("halves", fmt, tokens)
    ids, weights = to(np.zeros((tokens, 1), np.int32)), to(np.ones((tokens, 1), np.float32))
    got = qbn.moe_experts(make(parts, fmt), x.bfloat16().to(DEV), ids, weights).cpu().double().numpy()
    off = np.abs(got[:, 0] - (r - 64 * m))
    assert off.max() <= 1.0, "%g off at r = %d" % (off.max(), r[off.argmax()])
    assert (got[:, 1:] == 0).all()


@pytest.mark.parametrize("tokens", [1, 9])
def test_h_at_the_end_of_the_range(tokens):
    """A finite h whose upper part would round to infinity stays finite."""
    x = torch.zeros(tokens, 32)
    # h = 128 (2^121 - 2^111): past half the step from bfloat16's largest number, 2^128 - 2^120, to 2^128
    x[:, 0], x[:, 1], x[:, 2] = 128, 2.0 ** 121 - 2.0 ** 113, 2.0 ** 112 + 2.0 ** 111
    assert torch.equal(x.bfloat16().float(), x)
    rows = [(0, 0, 1), (32, 1, 1), (32, 2, 1)]
    one = np.full((1, 64, 1), 127, np.uint8)
    w2 = np.full((1, 32, 1), 127 - 64, np.uint8)
    parts = [one_hot(64, 32, rows)[None], one, None, one_hot(32, 32, [(i, 0, 1) for i in range(32)])[None], w2, None]
    ids, weights = to(np.zeros((tokens, 1), np.int32)), to(np.ones((tokens, 1), np.float32))
    say("end of the range", tokens)
    got = qbn.moe_experts(make(parts, "mxfp4"), x.bfloat16().to(DEV), ids, weights).cpu()
    assert (got == 2.0 ** 64).all()
