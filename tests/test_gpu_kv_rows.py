"""GPU: which rows of q, k and v are whose. Rows that no sequence has (before
cu[0], from cu[seqs] on) and calls without cu, against the references of
test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

import bit_block_quantized_nibble_amd as qbn
import kv_ref as R
from gpu_util import DEV, say
from test_gpu_kv_attention import FORMATS, random_cache, vectors

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seqs,each", [(2, 1), (2, 40), (70, 1), (70, 40)])
def test_append_leaves_rows_of_no_sequence_out(fmt, seqs, each):
    """cu starts after row 0 and ends before the last row: the rows outside it are
    written nowhere, above all not over a sequence's earlier tokens."""
    rng = np.random.default_rng(seqs + each)
    ps, heads, dim, row, before, after = 16, 2, 64, 8, 9, 5
    news = [each] * seqs
    lens = [n + 30 for n in news]
    pages = sum(-(-n // ps) for n in lens)
    table = R.torch_table(lens, ps, row, pages, rng)
    c = random_cache(fmt, pages, heads, ps, dim, None, junk=0x5A)
    want = [t.cpu() if t is not None else None for t in (c.k, c.v, c.k_scales, c.v_scales)]
    cu = before + np.concatenate([[0], np.cumsum(news)])
    x = [vectors(rng, int(cu[-1]) + after, heads, dim) for _ in range(2)]
    say("append", fmt, seqs, each)
    qbn.kv_append(c, x[0].to(DEV), x[1].to(DEV), table.to(DEV), ints(lens), ints(cu.tolist()))
    torch.cuda.synchronize()
    for which in (0, 1):
        code, scale = (None, None) if fmt == "bf16" else R.quantize(fmt, x[which].double().numpy())
        if fmt == "mxfp4":
            code = code[..., 0::2] | (code[..., 1::2] << 4)
        for b in range(seqs):
            for i in range(news[b]):
                pos, t = lens[b] - news[b] + i, int(cu[b]) + i
                page = int(table[b, pos // ps])
                want[which][0, page, :, pos % ps] = x[which][t] if code is None else torch.from_numpy(code[t])
                if code is not None:
                    want[which + 2][0, page, :, :, pos % ps] = torch.from_numpy(scale[t])
    for got, w, name in zip((c.k, c.v, c.k_scales, c.v_scales), want, ("k", "v", "k_scales", "v_scales")):
        if w is not None:
            assert torch.equal(got.cpu().view(torch.uint8), w.view(torch.uint8)), name
