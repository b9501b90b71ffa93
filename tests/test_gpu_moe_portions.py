"""GPU: calls of more tokens than the workspace holds at a time. Each portion sums in the
same order, so that like tokens have like bits wherever they stand, also in a last
portion of one or a few tokens. Inputs whose large terms cancel show another order."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import step_ref as S
from gpu_util import DEV, say
from test_gpu_moe import FORMATS, choice, make, to

pytestmark = pytest.mark.gpu


def cancelling(rng, fmt, tokens, experts, part, inter):
    """A layer and rows of three parts: large values, their negatives against the same
    weights, and ordinary ones."""
    c13, s13, f13, c2, s2, f2 = S.layer(rng, fmt, experts, 3 * part, inter)
    c13[..., part // 2:part] = c13[..., :part // 2]
    block = 32 if fmt == "mxfp4" else 16
    s13[..., part // block:2 * part // block] = s13[..., :part // block]
    big = rng.standard_normal((tokens, part)) * 10.0 ** rng.uniform(0, 3, (tokens, part))
    x = torch.from_numpy(np.concatenate([big, -big, rng.standard_normal((tokens, part))], 1).astype(np.float32))
    return make((c13, s13, f13, c2, s2, f2), fmt), x.to(torch.bfloat16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [257, 258, 263, 264, 270, 515])
def test_order_of_tokens_changes_no_bit(fmt, tokens):
    rng = np.random.default_rng(tokens)
    layer, x = cancelling(rng, fmt, tokens, 6, 352, 288)
    x = x.to(DEV)
    ids, weights = (to(a) for a in choice(rng, tokens, 6, 3))
    order = torch.arange(tokens - 1, -1, -1, device=DEV)  # the last portion's tokens come first
    say("order", fmt, tokens)
    out = qbn.moe_experts(layer, x, ids, weights)
    assert torch.isfinite(out).all()
    assert torch.equal(qbn.moe_experts(layer, x[order], ids[order], weights[order]), out[order])


@pytest.mark.parametrize("tokens", [257, 263, 520])
def test_like_tokens_have_like_rows(tokens):
    rng = np.random.default_rng(tokens)
    layer, x = cancelling(rng, "mxfp4", 1, 4, 1376, 1056)
    ids, weights = (to(np.repeat(a, tokens, 0)) for a in choice(rng, 1, 4, 4))
    say("like", tokens)
    out = qbn.moe_experts(layer, x.to(DEV).expand(tokens, -1).contiguous(), ids, weights)
    assert torch.equal(out, out[:1].expand(tokens, -1))
