"""GPU: choices for more tokens than the workspace holds at a time: like tokens have like
experts and weights, bit by bit, also in a last portion of one or a few tokens."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
from gpu_util import DEV, say
from test_gpu_moe import router

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [4097, 4098, 4099, 4112, 8193])
@pytest.mark.parametrize("experts,hidden", [(20, 1024), (130, 2080)])
@pytest.mark.parametrize("normalize", [True, False])
def test_choice_of_like_tokens(tokens, experts, hidden, normalize):
    """Logits that are what binary64 sums of cancelling terms leave: another order, other logits."""
    rng = np.random.default_rng(hidden)
    half = hidden // 2
    w = rng.standard_normal((experts, half)) * 2.0 ** rng.uniform(-10, 46, (experts, half))
    w = torch.from_numpy(np.concatenate([w, -w[:, rng.permutation(half)]], 1).astype(np.float32)).to(torch.bfloat16)
    x = torch.ones(tokens, hidden, dtype=torch.bfloat16)
    say("choice", tokens, experts, hidden)
    ids, weights = qbn.moe_route(router(w, 3, normalize=normalize), x.to(DEV))
    assert torch.equal(ids, ids[:1].expand(tokens, -1)) and torch.equal(weights, weights[:1].expand(tokens, -1))
