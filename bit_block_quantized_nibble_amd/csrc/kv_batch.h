// The batch of a paged cache's call from its tensors (host code).
#pragma once

#include "../../include/qbn_kv.h"
#include "bind.h"

namespace qcall {

inline qbn_kv_batch batch(int64_t dev, int64_t tokens, const at::Tensor &table, const at::Tensor &lens, PyObject *cu) {
    typed(table, at::kInt, "torch.int32", "table");
    if (table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
        refuse(PyExc_ValueError, "table must be [seqs][row] with contiguous rows");
    if (index_of(table) != dev) elsewhere(table, "table");
    qbn_kv_batch b;
    b.seqs = table.size(0), b.tokens = tokens, b.row = table.size(1);
    b.row_stride = b.seqs > 1 ? table.stride(0) : b.row;
    b.table = (const int32_t *)table.data_ptr();
    b.cu = nullptr;
    if (cu == Py_None && tokens != b.seqs)
        refuse(PyExc_ValueError, "%lld tokens for %lld sequences: one each is wanted without cu", (long long)tokens, (long long)b.seqs);
    b.lens = ints(lens, b.seqs, dev, "lens");
    if (cu != Py_None) b.cu = ints(tensor(cu, "cu"), b.seqs + 1, dev, "cu");
    return b;
}

}  // namespace qcall
