// Writing elements of the paged key-value cache: rounding to its formats.
#pragma once

#include "kv_device.h"

namespace qbn {
namespace kv {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// Writes eight elements at dst (16, 8 or 4 bytes); four lanes of a quad have the
// 32 of a block. Returns the block's shared exponent (MX formats). All four lanes
// call it together.
template <int F>
__device__ __forceinline__ int put8(uint8_t *dst, float (&x)[8]) {
    if constexpr (F == BF16) {
        *reinterpret_cast<u32x4 *>(dst) =
            u32x4{pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
        return 0;
    } else {
        uint32_t top = 0;  // magnitudes as bit patterns order like the values
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
        top = max(top, dpp_u32<0xB1>(top));  // quad_perm [1,0,3,2]
        top = max(top, dpp_u32<0x4E>(top));  // quad_perm [2,3,0,1]: the four lanes of the block
        constexpr int EMAX = F == FP8 ? 8 : 2;
        int e = (int)(top >> 23) - 127 - EMAX;
        e = e < -127 ? -127 : (e > 127 ? 127 : e);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_ldexpf(x[i], -e);
        if constexpr (F == FP8) {
            typedef short v2s __attribute__((ext_vector_type(2)));
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __builtin_fminf(__builtin_fmaxf(x[i], -448.0f), 448.0f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v2s p = {0, 0};
                p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, x[4 * i], x[4 * i + 1], 1.0f, false);
                p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, x[4 * i + 2], x[4 * i + 3], 1.0f, true);
                w[i] = __builtin_bit_cast(uint32_t, p);
            }
            *reinterpret_cast<u32x2 *>(dst) = u32x2{w[0], w[1]};
        } else {
            uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], 1.0f, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], 1.0f, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], 1.0f, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], 1.0f, 3);
            *reinterpret_cast<uint32_t *>(dst) = w;
        }
        return e;
    }
}

}  // namespace kv
}  // namespace qbn
