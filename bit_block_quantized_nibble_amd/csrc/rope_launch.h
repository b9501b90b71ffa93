// Launch entry points of the rotation by positions. Arguments have been validated
// by the C-ABI layer (kv_api.hip).
#pragma once

#include "kv_launch.h"
#include "qbn_rope.h"

namespace qbn {

struct KvRowsOut {  // as KvRows, to be written
    void *p;
    int64_t token_stride, head_stride;
};

hipError_t launch_rope(const qbn_rotation &r, int64_t tokens, int heads, int dim, const int32_t *positions,
                       const KvRows &x, const KvRowsOut &out, int dtype, hipStream_t s);

hipError_t launch_kv_append_rope(const qbn_kv_cache &c, int64_t layer, const qbn_kv_batch &b, const qbn_rotation &r,
                                 int q_heads, const KvRows &q, const KvRowsOut &out, const KvRows &k, const KvRows &v,
                                 int dtype, hipStream_t s);

}  // namespace qbn
