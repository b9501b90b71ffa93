"""Host-side limits of the paged cache's calls: sizes that no launch can have are
refused before anything is enqueued. No pointer below is dereferenced."""
import ctypes

import pytest

from bit_block_quantized_nibble_amd import kv

A = 0x10000
SHAPE = 4


def call(decode, seqs, tokens, heads, q_heads, row, cu=None, scale=0.1):
    lib = kv._kv()
    c = ctypes.byref(kv._CCache(16, heads, 64, 16, 1, 8, A, A, None, None))
    b = ctypes.byref(kv._CBatch(seqs, tokens, row, row, A, A, cu))
    f = lib.qbn_kv_attention_decode if decode else lib.qbn_kv_attention_prefill
    got = lib.qbn_kv_attention_workspace(c, b, q_heads, 0, 0, int(decode))
    return got, f(c, 0, b, q_heads, A, 64 * q_heads, 64, scale, 0, 0, A, A, A, 1 << 60, None)


@pytest.mark.parametrize("decode,seqs,heads,q_heads,row", [
    (True, 1 << 18, 64, 64, 1),         # 2^24 pairs of one workgroup
    (True, 1 << 18, 64, 64, 4096),      # as many, cut in pieces
    (True, 1 << 20, 1, 64, 4096),       # 2^20 pairs, but 2^26 rows to join, four a workgroup
    (True, 1 << 18, 4096, 4096, 16),
    (False, 1 << 20, 32, 32, 1),        # 2^25 tiles of 256 threads
    (False, 1 << 18, 4096, 4096, 4096),
])
def test_grids_of_2_to_the_32_threads_are_refused(decode, seqs, heads, q_heads, row):
    assert call(decode, seqs, seqs, heads, q_heads, row) == (-1, SHAPE)


def test_many_empty_sequences_are_refused_in_prefill():
    assert call(False, 1 << 20, 16, 4096, 4096, 1, cu=A) == (-1, SHAPE)


@pytest.mark.parametrize("decode", [True, False])
def test_the_most_sequences_fit(decode):
    c = ctypes.byref(kv._CCache(16, 8, 64, 16, 1, 8, A, A, None, None))
    b = ctypes.byref(kv._CBatch(1 << 20, 1 << 20, 4096, 4096, A, A, None))
    assert kv._kv().qbn_kv_attention_workspace(c, b, 32, 0, 0, int(decode)) >= 0


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_scales_that_pass_binary32_in_base_2_are_refused(decode, scale):
    """scale * log2 e would be infinite, and 0 times it NaN. (Without tokens there
    is nothing to launch.)"""
    assert call(decode, 4, 4, 2, 4, 1, scale=scale)[1] == SHAPE
    assert call(decode, 0, 0, 2, 4, 1, scale=scale)[1] == SHAPE
    assert call(decode, 0, 0, 2, 4, 1, scale=2.3e38)[1] == 0
