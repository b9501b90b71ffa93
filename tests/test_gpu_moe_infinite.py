"""GPU: MXFP4 weights beyond bfloat16's largest number (scale bytes 253 and 254): what
they enter is infinite or NaN, whatever the length of the row, and nothing else is."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import step_ref as S
from gpu_util import DEV, say
from test_gpu_moe import check_experts, make, to

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("byte", [253, 254])
@pytest.mark.parametrize("tokens", [2, 70])
@pytest.mark.parametrize("k", [32, 96, 256, 288, 512])
def test_weights_beyond_the_range(byte, tokens, k):
    rng = np.random.default_rng(k + tokens)
    parts = S.layer(rng, "mxfp4", 3, k, k)
    good = [None if p is None else p.copy() for p in parts]
    x = S.bf16(rng, tokens, k)
    assert (x != 0).all()
    # the second product of expert 1, output row 5, the last block; the first product of expert 2, an up row
    parts[4][1, 5, -1], parts[3][1, 5, -16:] = byte, 0x77
    parts[1][2, k + 3, -1], parts[0][2, k + 3, -16:] = byte, 0x77
    ids = (np.arange(tokens) % 3).astype(np.int32)[:, None]
    weights = np.ones((tokens, 1), np.float32)
    say("beyond", byte, tokens, k)
    got = qbn.moe_experts(make(parts, "mxfp4"), x.to(DEV), to(ids), to(weights)).cpu()
    bad = ~torch.isfinite(got)
    want = torch.zeros(tokens, k, dtype=torch.bool)
    want[1::3, 5], want[2::3] = True, True
    assert torch.equal(bad, want)
    fine = np.arange(0, tokens, 3)
    check_experts(got[fine], x[fine], ids[fine], weights[fine], good, "mxfp4")
    rest = [i for i in range(k) if i != 5]
    out, tol = S.experts(x[1::3].double().numpy(), ids[1::3], weights[1::3].astype(np.float64),
                         S.decode("mxfp4", good[0], good[1]), S.decode("mxfp4", good[3], good[4]))
    assert (np.abs(got[1::3].double().numpy() - out) <= tol)[:, rest].all()
