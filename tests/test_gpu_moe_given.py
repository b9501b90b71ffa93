"""GPU: what a call is given to write into is what it returns and what holds the results."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import step_ref as S
from gpu_util import DEV, say
from test_gpu_moe import FORMATS, make, router

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [1, 3, 40, 300])
def test_given_outputs_hold_the_results(fmt, tokens):
    rng = np.random.default_rng(tokens)
    layer = make(S.layer(rng, fmt, 6, 96, 64), fmt, router(S.bf16(rng, 6, 96, gain=0.3), 2))
    x = S.bf16(rng, tokens, 96).to(DEV)
    want = qbn.moe(layer, x)

    def given():
        wide = torch.full((tokens, 120), 9.0, dtype=torch.bfloat16, device=DEV)
        ids = torch.full((tokens, 2), -7, dtype=torch.int32, device=DEV)
        return wide, wide[:, 16:112], ids, torch.full((tokens, 2), -7.0, device=DEV)

    def same(got, into):
        for g, t, w in zip(got, into, want):
            assert g.data_ptr() == t.data_ptr() and g.shape == t.shape and g.stride() == t.stride()
            assert torch.equal(t, w)

    say("given", fmt, tokens)
    wide, out, ids, weights = given()
    same(qbn.moe(layer, x, out=out, ids=ids, weights=weights), (out, ids, weights))
    assert (wide[:, :16] == 9).all() and (wide[:, 112:] == 9).all()
    wide, out, ids, weights = given()
    got = qbn.moe_route(layer.router, x, ids=ids, weights=weights)
    same((want[0],) + tuple(got), (want[0], ids, weights))
    got = qbn.moe_experts(layer, x, ids, weights, out=out)
    same((got, ids, weights), (out, ids, weights))
    assert (wide[:, :16] == 9).all() and (wide[:, 112:] == 9).all()
