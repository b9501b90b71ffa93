// Launch entry points of the paged key-value cache. Arguments have been
// validated by the C-ABI layer (kv_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qbn_kv.h"

namespace qbn {

struct KvRows {  // [token][head] vectors of head_dim elements, strides in elements
    const void *p;
    int64_t token_stride, head_stride;
};

hipError_t launch_kv_append(const qbn_kv_cache &c, int64_t layer, const qbn_kv_batch &b, const KvRows &k,
                            const KvRows &v, int dtype, hipStream_t s);

// Bytes of a call's workspace; -1 where a launch would pass the 2^32 threads of a grid.
int64_t kv_decode_workspace(const qbn_kv_cache &c, const qbn_kv_batch &b, int q_heads, int window, int sinks);
hipError_t launch_kv_decode(const qbn_kv_cache &c, int64_t layer, const qbn_kv_batch &b, int q_heads, const KvRows &q,
                            float scale, int window, int sinks, void *out, float *lse, void *ws, hipStream_t s);

int64_t kv_prefill_workspace(const qbn_kv_cache &c, const qbn_kv_batch &b, int q_heads, int window, int sinks);
hipError_t launch_kv_prefill(const qbn_kv_cache &c, int64_t layer, const qbn_kv_batch &b, int q_heads, const KvRows &q,
                             float scale, int window, int sinks, void *out, float *lse, void *ws, hipStream_t s);

int64_t kv_pool_workspace(const qbn_kv_pool &p, int64_t count);
hipError_t launch_kv_reserve(const qbn_kv_pool &in, const qbn_kv_pool &out, int64_t count, const int32_t *rows,
                             const int32_t *tokens, int32_t *status, void *ws, hipStream_t s);
hipError_t launch_kv_fork(const qbn_kv_cache &c, const qbn_kv_pool &in, const qbn_kv_pool &out, int64_t count,
                          const int32_t *parents, const int32_t *children, int32_t *status, void *ws, hipStream_t s);
hipError_t launch_kv_free(const qbn_kv_pool &in, const qbn_kv_pool &out, int64_t count, const int32_t *rows,
                          int window, int sinks, hipStream_t s);
hipError_t launch_kv_compact(const qbn_kv_cache &c, const qbn_kv_pool &in, const qbn_kv_pool &out, int32_t *live,
                             void *ws, hipStream_t s);

}  // namespace qbn
