// Launch entry points of the experts' layer. Arguments have been validated by the
// C-ABI layer (moe_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qbn_moe.h"

namespace qbn {

int64_t moe_route_workspace(const qbn_moe_router &r, int64_t tokens);
hipError_t launch_moe_route(const qbn_moe_router &r, int64_t tokens, const void *x, int64_t x_stride, int32_t *ids,
                            float *weights, void *ws, hipStream_t s);

int64_t moe_experts_workspace(const qbn_moe_weights &e, int64_t tokens, int top_k);
hipError_t launch_moe_experts(const qbn_moe_weights &e, int64_t tokens, int top_k, const void *x, int64_t x_stride,
                              const int32_t *ids, const float *weights, void *out, int64_t out_stride, void *ws,
                              hipStream_t s);

}  // namespace qbn
