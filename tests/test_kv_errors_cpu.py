"""Errors that torch raises inside the paged cache's calls: with torch's types and
words, as from torch's own functions. Without a GPU."""
import pytest
import torch

from bit_block_quantized_nibble_amd import kv

A = 0x10000
K, T, L = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)


@pytest.mark.filterwarnings("ignore:Sparse CSR")
@pytest.mark.parametrize("decode", [True, False])
def test_errors_of_torch_come_through_without_a_backtrace(decode):
    cache = bytes(kv._CCache(16, 2, 64, 16, 1, 8, A, A, None, None))
    odd = torch.zeros(4, 4).to_sparse_csr()
    with pytest.raises(RuntimeError) as direct:
        odd.is_contiguous()
    with pytest.raises(RuntimeError) as ours:
        kv._call().attention(decode, cache, -1, K, None, T, L, 0, 0, 0.1, 0, None, None, odd)
    assert type(ours.value) is type(direct.value)
    assert "Exception raised from" not in str(ours.value)
