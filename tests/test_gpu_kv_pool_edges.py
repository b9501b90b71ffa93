"""GPU: bookkeeping of pools whose rows have no entries, or that have no slots:
what is written into other tables is all of the pool."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v, np.int32), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("seqs,row", [(3, 0), (0, 4), (0, 0)])
@pytest.mark.parametrize("what", ["reserve", "free", "fork", "compact"])
def test_pools_without_entries(seqs, row, what):
    pages, ps = 70, 16
    refs = np.arange(pages) % 3
    pool = qbn.KVPool(torch.zeros((seqs, row), dtype=torch.int32, device=DEV), ints([0] * seqs), ints(refs), ps)
    out = qbn.KVPool.like(pool)
    for t in (out.table, out.lens, out.refs):
        t.fill_(77)
    c = qbn.KVCache.empty("mxfp4", 1, pages, 1, ps, 64, device=DEV)
    rows, none = ints(list(range(seqs))), ints([0] * seqs)
    say(what, seqs, row)
    if what == "reserve":
        assert int(qbn.kv_reserve(pool, rows, none, out=out)) == -1
    elif what == "free":
        qbn.kv_free(pool, rows, out=out)
    elif what == "fork":
        n = 2 if seqs else 0
        assert int(qbn.kv_fork(c, pool, rows[:n] * 0, rows[:n] + 1, out=out)) == -1
    else:
        assert int(qbn.kv_compact(c, pool, out=out)) == int((refs > 0).sum())
        total, refs = refs.sum(), out.refs.cpu().numpy()
        assert (refs[:46] > 0).all() and (refs[46:] == 0).all() and refs.sum() == total
    torch.cuda.synchronize()
    assert out.lens.cpu().tolist() == [0] * seqs
    assert np.array_equal(out.refs.cpu().numpy(), refs)
