"""GPU: what the paged cache's calls raise where memory runs out."""
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def test_running_out_of_memory_raises_torchs_type():
    """A server catches torch.OutOfMemoryError to give pages back. The output asked
    for has 512 GiB, more than the device; its query is one row repeated."""
    c = qbn.KVCache.empty("bf16", 1, 2, 1, 16, 256, device=DEV)
    q = torch.zeros(1, 1, 256, dtype=torch.bfloat16, device=DEV).expand(1 << 24, 64, 256)
    table, lens = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1 << 24], dtype=torch.int32, device=DEV)
    say("out of memory")
    with pytest.raises(torch.OutOfMemoryError):
        qbn.kv_attention_prefill(c, q, cu, table, lens)
    out, lse = qbn.kv_attention_prefill(c, q[:3], cu * 0, table, lens)  # and goes on
    assert (out == 0).all() and (lse == -float("inf")).all()
