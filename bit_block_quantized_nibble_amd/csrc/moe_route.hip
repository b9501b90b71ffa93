// Choosing the experts of each token: logits, the top_k of them, their weights.
//
// Which expert comes next may hang on the last bit of a logit, so the sums are
// binary64: products of bfloat16 values are exact, and the order of a sum of
// thousands of them then moves it by 1e-16 instead of 1e-7. The vector units do a
// binary64 fma at the rate of an unpacked binary32 one, and the matrix cores as many: 72 and 77 TFLOP/s
// measured, 64 cycles for a step of 16 x 16 x 4.
//
// Few tokens: a workgroup per expert, its row read once and multiplied with each
// token's; bound by latency. More: 16 tokens by 16 experts a workgroup on the
// matrix cores, k split over its waves; then a wave per token finds the best one after the other.
//
// One token, 128 experts, 4096: 2.7 us and 3.9 for the choice, of which 2.4 each are an empty
// kernel's. 1999 tokens, 64 experts, 2048: 14.8 us, where the products alone take 6.8 and a launch 2.4; choice 4.4. The matrix
// cores are busy for 57 % of the kernel's cycles: a wave has 32 products, each after the one before, in four runs that each
// follow their loads, and waits for those in 42 % of its cycles.
// Split over k, 256 tokens of 128 experts (4096) take 9.3 us, else 14.5.
#include "moe_launch.h"
#include "rope_device.h"

#include <algorithm>

namespace qbn {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int64_t kPortion = 4096;  // tokens whose logits the workspace holds at a time
// Tokens of the vector form: 128 experts, 4096, take 2.9 us for one token and 3.2 for two, 4.0 in tiles of
// 16 tokens; four take 4.0 either way.
constexpr int kFew = 2;
constexpr int64_t kParts = 8;       // of the hidden size, at most

struct Args {
    const __bf16 *x, *w;
    double *logits;  // [parts][tokens][experts], without the bias
    const float *bias;
    int32_t *ids;
    float *weights;
    int64_t xs;
    int tokens, experts, hidden, top, normalize, parts;
};

// The sum over a wave's lanes, in all of them.
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Numbers as unsigned words of the same order, all of them above 0; NaN as -inf.
__device__ __forceinline__ uint64_t ordered(double v) {
    if (v != v) v = -__builtin_huge_val();
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 is 0
    return b ^ (b >> 63 ? ~(uint64_t)0 : (uint64_t)1 << 63);
}
__device__ __forceinline__ double number(uint64_t b) {
    return __builtin_bit_cast(double, b ^ (b >> 63 ? (uint64_t)1 << 63 : ~(uint64_t)0));
}

// The largest over a wave's lanes, the same in all of them.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    const auto step = [](uint32_t x, int y) { return max(x, (uint32_t)y); };
    v = step(v, kv::dpp_i32<0x111, 0xF>((int)v));  // shifts within rows of 16, then rows into the next
    v = step(v, kv::dpp_i32<0x112, 0xF>((int)v));  // (lanes without a source read 0)
    v = step(v, kv::dpp_i32<0x114, 0xF>((int)v));
    v = step(v, kv::dpp_i32<0x118, 0xF>((int)v));
    v = step(v, kv::dpp_i32<0x142, 0xA>((int)v));
    v = step(v, kv::dpp_i32<0x143, 0xC>((int)v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// Of words of 64 bits: their upper halves decide, and where several lanes have the largest, the lower.
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    const uint32_t hi = wave_max((uint32_t)(v >> 32));
    const bool mine = (uint32_t)(v >> 32) == hi;
    const uint64_t m = __ballot(mine);
    const uint32_t lo = m & (m - 1) ? wave_max(mine ? (uint32_t)v : 0)
                                    : (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, __builtin_ctzll(m));
    return (uint64_t)hi << 32 | lo;
}

template <int T>
__global__ __launch_bounds__(256) void k_logits_few(Args a) {
    __shared__ double part[4][T];
    const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double sum[T] = {};
    for (int k = threadIdx.x * 8; k < a.hidden; k += 256 * 8) {
        float w[8], x[8];
        rope::floats(rope::load8(a.w + (int64_t)e * a.hidden + k), w);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            rope::floats(rope::load8(a.x + min(t, a.tokens - 1) * a.xs + k), x);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[t] = __builtin_fma((double)w[i], (double)x[i], sum[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const double s = wave_sum(sum[t]);
        if (lane == 0) part[wave][t] = s;
    }
    __syncthreads();
    if ((int)threadIdx.x < T && (int)threadIdx.x < a.tokens) {
        a.logits[(int64_t)threadIdx.x * a.experts + e] =
            (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
    }
}

// 16 tokens x 16 experts. A wave's k come in pieces of 32, of which the lanes of a
// quarter (16 lanes) have eight in a row each: which k a product step takes is
// free, as long as both operands agree. Of a part of k: blockIdx.y.
constexpr int kWaves = 16;
__global__ __launch_bounds__(kWaves * 64) void k_logits(Args a) {
    __shared__ double part[kWaves][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quarter = lane >> 4;
    const int tiles = (a.experts + 15) / 16;
    const int t0 = (int)(blockIdx.x / tiles) * 16, e0 = (int)(blockIdx.x % tiles) * 16;
    const __bf16 *x = a.x + (int64_t)min(t0 + row, a.tokens - 1) * a.xs + quarter * 8;
    const __bf16 *w = a.w + (int64_t)min(e0 + row, a.experts - 1) * a.hidden + quarter * 8;
    f64x4 acc = {0, 0, 0, 0};
    for (int k = (wave * a.parts + blockIdx.y) * 32; k < a.hidden; k += kWaves * a.parts * 32) {
        float u[8], v[8];
        rope::floats(rope::load8(x + k), u);
        rope::floats(rope::load8(w + k), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)u[i], (double)v[i], acc, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][(quarter + 4 * i) * 16 + row] = acc[i];  // token quarter + 4 i, expert row
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += kWaves * 64) {
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < kWaves; ++j) s += part[j][i];
        const int t = t0 + i / 16, e = e0 + i % 16;
        if (t < a.tokens && e < a.experts) a.logits[((int64_t)blockIdx.y * a.tokens + t) * a.experts + e] = s;
    }
}

// A wave per token; lane l looks at experts l, l + 64, ... (EACH of them).
template <int EACH>
__global__ __launch_bounds__(256) void k_choose(Args a) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.tokens) return;
    uint64_t key[EACH];
    double v[EACH];
    bool nan = false;
#pragma unroll
    for (int j = 0; j < EACH; ++j) v[j] = a.bias ? (double)a.bias[min(lane + 64 * j, a.experts - 1)] : 0.0;
    constexpr int AHEAD = EACH <= 4 ? 8 : 2;  // loads sent together: one after another, they cost a microsecond each
    for (int p0 = 0; p0 < a.parts; p0 += AHEAD) {
        double u[AHEAD][EACH];
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
#pragma unroll
            for (int j = 0; j < EACH; ++j)
                u[p][j] = a.logits[((int64_t)min(p0 + p, a.parts - 1) * a.tokens + t) * a.experts +
                                   min(lane + 64 * j, a.experts - 1)];
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
#pragma unroll
            for (int j = 0; j < EACH; ++j) v[j] += p0 + p < a.parts ? u[p][j] : 0.0;
    }
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        key[j] = lane + 64 * j < a.experts ? ordered(v[j]) : 0;
        nan = nan || v[j] != v[j];
    }
    nan = __ballot(nan) != 0;
    int id = 0;
    double mine = 0.0, best = 0.0;  // its logit, and the largest
    for (int r = 0; r < a.top; ++r) {
        uint64_t top = key[0];
#pragma unroll
        for (int j = 1; j < EACH; ++j) top = key[j] > top ? key[j] : top;
        top = wave_max(top);
        int e = 0x7FFFFFFF;
#pragma unroll
        for (int j = EACH - 1; j >= 0; --j) {  // the lowest number among equal ones
            const uint64_t m = __ballot(key[j] == top);
            if (m) e = 64 * j + __builtin_ctzll(m);
        }
#pragma unroll
        for (int j = 0; j < EACH; ++j)
            if (e == lane + 64 * j) key[j] = 0;
        if (lane == r) id = e, mine = number(top);
        if (r == 0) best = number(top);
    }
    double total = 0.0;
    if (!a.normalize) {
        double s = 0.0;
        for (int j = 0; j < EACH; ++j)
            if (lane + 64 * j < a.experts) s += exp((v[j] != v[j] ? -__builtin_huge_val() : v[j]) - best);
        total = wave_sum(s);
    }
    const double p = lane < a.top ? exp(mine - best) : 0.0;
    if (a.normalize) total = wave_sum(p);
    if (nan) total = __builtin_nan("");
    if (lane < a.top) {
        a.ids[(int64_t)t * a.top + lane] = id;
        a.weights[(int64_t)t * a.top + lane] = (float)(p / total);
    }
}


// Where there are fewer tiles of 16 x 16 than compute units, k is split over them too, a piece of 32 (eight
// products, one after the other) for each wave at least.
int parts_of(const qbn_moe_router &r, int64_t tokens) {
    const int64_t tiles = (tokens + 15) / 16 * ((r.experts + 15) / 16), most = (r.hidden + 511) / 512;
    const int64_t parts = tokens <= kFew ? 1 : std::min<int64_t>({kParts, 256 / tiles, most});
    return (int)std::max<int64_t>(parts, 1);
}

}  // namespace

// No less for more tokens: parts * tiles <= 256 where parts > 1.
int64_t moe_route_workspace(const qbn_moe_router &r, int64_t tokens) {
    const int64_t n = std::min(tokens, kPortion), split = 256 * 16 / ((r.experts + 15) / 16);
    return 8 * r.experts * std::max(n, std::min(kParts * n, split));
}

hipError_t launch_moe_route(const qbn_moe_router &r, int64_t tokens, const void *x, int64_t x_stride, int32_t *ids,
                            float *weights, void *ws, hipStream_t s) {
    Args a = {};
    a.w = (const __bf16 *)r.weight, a.bias = r.bias, a.logits = (double *)ws, a.xs = x_stride;
    a.experts = r.experts, a.hidden = r.hidden, a.top = r.top_k, a.normalize = r.normalize;
    // Form and parts are the whole call's: the last portion's logits are summed in the same order as the others'.
    const bool few = tokens <= kFew;
    a.parts = parts_of(r, tokens);
    for (int64_t at = 0; at < tokens; at += kPortion) {
        a.tokens = (int)std::min(tokens - at, kPortion);
        a.x = (const __bf16 *)x + at * x_stride, a.ids = ids + at * r.top_k, a.weights = weights + at * r.top_k;
        if (few) {
            (a.tokens == 1 ? k_logits_few<1> : k_logits_few<2>)<<<r.experts, 256, 0, s>>>(a);
        } else {
            const int tiles = (a.tokens + 15) / 16 * ((a.experts + 15) / 16);
            k_logits<<<dim3(tiles, a.parts), kWaves * 64, 0, s>>>(a);
        }
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int blocks = (a.tokens + 3) / 4, each = (r.experts + 63) / 64;
        (each <= 1 ? k_choose<1> : each <= 2 ? k_choose<2> : each <= 4 ? k_choose<4> : each <= 8 ? k_choose<8> : k_choose<16>)
            <<<blocks, 256, 0, s>>>(a);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qbn
