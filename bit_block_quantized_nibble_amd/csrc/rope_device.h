// The rotation by positions, device side (gfx950 only): shared by the kernel that
// turns vectors in memory and the one that turns them on the way into the cache.
#pragma once

#include "kv_device.h"
#include "qbn_rope.h"

namespace qbn {
namespace rope {

struct Rotation {
    const uint64_t *turns;  // per pair: 2^64 of a turn per position
    int rot;
    float factor;
};

// Bits 32 to 63 of p * turns in 64-bit arithmetic that wraps: the angle without
// its whole turns, in units of 2^-32 turns. The product is of the unsigned p; a
// negative one is p + 2^32, and 2^32 * turns adds the low word of turns up here.
__device__ __forceinline__ uint32_t angle_of(int p, u32x2 turns) {
    const uint32_t u = (uint32_t)p;
    return __umulhi(u, turns.x) + u * turns.y - (p < 0 ? turns.x : 0u);
}

// factor * cos and factor * sin of an angle in 2^-32 turns. The nearest quarter turn
// is taken off exactly, what is left lies in [-pi/4, pi/4], where the Taylor series
// to a^9 and a^10 are off by 2e-9 and 1e-10: below half a unit of binary32. What a binary32
// angle lacks goes into the terms before the last sum, so that a turned number's rounding to
// fewer bits is hardly ever another one: sines are 0.19 units of 2^-24 off in the mean square (0.33
// without), where correctly rounded ones are 0.19, cosines 0.31 (0.35), and 0.29.
__device__ __forceinline__ void cos_sin(uint32_t angle, float factor, float &c, float &s) {
    const uint32_t quarter = (angle + 0x20000000u) >> 30;
    const int left = (int)(angle - (quarter << 30));
    const float f = (float)left, unit = 1.4629180792671596e-9f;  // 2 pi / 2^32, less the next line's rest
    const float a = f * unit, q = a * a;
    float rest = __builtin_fmaf(f, -4.070940267922164e-17f, __builtin_fmaf(f, unit, -a));
    rest = __builtin_fmaf((float)(left - (int)f), unit, rest);  // what a lacks
    float sn = __builtin_fmaf(q, 2.7557319223985893e-6f, -1.984126984126984e-4f);
    sn = __builtin_fmaf(q, sn, 8.333333333333333e-3f);
    sn = __builtin_fmaf(q, sn, -1.6666666666666666e-1f);
    sn = a + __builtin_fmaf(q * a, sn, rest * __builtin_fmaf(q, -0.5f, 1.0f));
    float cs = __builtin_fmaf(q, -2.755731922398589e-7f, 2.48015873015873e-5f);
    cs = __builtin_fmaf(q, cs, -1.388888888888889e-3f);
    cs = __builtin_fmaf(q, cs, 4.1666666666666664e-2f);
    cs = __builtin_fmaf(q, cs, -0.5f);
    cs = 1.0f + __builtin_fmaf(q, cs, -(rest * a));
    const bool swap = quarter & 1u;
    c = (swap ? sn : cs) * factor;
    s = (swap ? cs : sn) * factor;
    c = __uint_as_float(__float_as_uint(c) ^ (((quarter + 1u) & 2u) << 30));  // quarters 1 and 2: negative
    s = __uint_as_float(__float_as_uint(s) ^ ((quarter & 2u) << 30));         // quarters 2 and 3
}

// a cos - b sin, b cos + a sin.
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = __builtin_fmaf(a, c, -(b * s));
    b = __builtin_fmaf(b, c, a * s);
    a = x;
}

// Eight elements from or to memory (16-byte aligned) as binary32.
template <typename T>
struct Eight {
    u32x4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T *p) {
    Eight<T> e;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) e.w[i] = ld16((const uint8_t *)p + 16 * i);
    return e;
}
__device__ __forceinline__ void floats(const Eight<float> &e, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(e.w[i / 4][i % 4]);
}
__device__ __forceinline__ void floats(const Eight<__bf16> &e, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(e.w[0][i] << 16);
        x[2 * i + 1] = __uint_as_float(e.w[0][i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        *reinterpret_cast<u32x4 *>(p + 4 * i) =
            u32x4{__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                  __float_as_uint(x[4 * i + 3])};
}
__device__ __forceinline__ void store8(__bf16 *p, const float (&x)[8]) {
    *reinterpret_cast<u32x4 *>(p) =
        u32x4{kv::pack2(x[0], x[1]), kv::pack2(x[2], x[3]), kv::pack2(x[4], x[5]), kv::pack2(x[6], x[7])};
}

// A lane's 16 elements of a head, the same in every head that it comes to: eight
// whole pairs where they turn (so that a vector can be turned in its place, by
// whatever order the lanes come in), 16 in a row where not.
struct Lane16 {
    int first, second;  // where its two runs of eight start
    bool turns;
};
template <bool HALF>
__device__ __forceinline__ Lane16 lane16(int group, int rot) {
    const bool turns = group < rot / 16;
    if (HALF && turns) return {8 * group, 8 * group + rot / 2, true};
    return {16 * group, 16 * group + 8, turns};
}

// Cosine and sine of the lane's eight pairs at a position.
__device__ __forceinline__ void spin8(const u32x2 (&turns)[8], float factor, int pos, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cos_sin(angle_of(pos, turns[i]), factor, c[i], s[i]);
}
__device__ __forceinline__ void load_turns(const Rotation &r, int pair, u32x2 (&turns)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const u32x4 w = ld16(r.turns + pair + 2 * i);
        turns[2 * i] = u32x2{w.x, w.y};
        turns[2 * i + 1] = u32x2{w.z, w.w};
    }
}
template <bool HALF>
__device__ __forceinline__ void turn16(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
    if constexpr (HALF) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(a[i], b[i], c[i], s[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn(a[2 * i], a[2 * i + 1], c[i], s[i]);
            turn(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
        }
    }
}

}  // namespace rope
}  // namespace qbn
