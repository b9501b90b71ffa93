// The experts' layer over 4-bit weights.
//
//   out_t = sum_j w_tj W2[e] (silu(Wg[e] x_t) * (Wu[e] x_t)),  e = ids[t][j]
// An assignment a = t * top_k + j is a token's j-th expert. Bound by the weights'
// bytes: each of a layer's active experts is read once for up to 64 of its assignments in the first
// product and 32 in the second, and again for more, and for each 256 tokens.
// So the weights go from memory to registers with nothing in between, are expanded
// there to bfloat16 (exactly) and multiplied on the matrix cores with the tokens as
// columns, 16 of them at the price of one.
//
// A lane's 16-byte load has 32 consecutive elements of a weight row, one MXFP4
// block or two of NVFP4, and the four 8-element words of it are the operands of four
// product steps: which k a step takes is free as long as the columns agree, and
// they have the same 8 elements each in one 16-byte load of x.
//
// First kernel: h for each assignment, from 16 gate rows and the 16 up rows beside them.
// h goes on as two bfloat16 values, the nearest one and the rest: one alone would round it
// by 2^-8, as much as the output's own rounding. Second kernel: the same products with
// W2. Where tokens are few, a workgroup has 16 output rows of all of them and adds up the
// tokens' experts itself; else the assignments' results go to memory and one more kernel
// adds them, in the order of a token's choices: the same bits every time.
//
// One token, 8 of 64 experts, 4096 x 1536, MXFP4: 13.5 and 9.2 us for 53 and 27 MB, bound by chains
// of dependent loads (of the first kernel's, 8 are the codes' way). 256 tokens, 8 of 128 such experts: 178 us
// for 856 MB, 4.8 TB/s, a large copy's rate and what its loads take alone; 127 for 428 MB, beside which
// the columns, two parts of h, are another 201 MB for its 16 groups of rows (5.4 million line requests in
// all, of which 3.1 are codes; a request in nine is met by the second cache), all through LDS.
#include "kv_device.h"
#include "moe_launch.h"

#include <algorithm>

namespace qbn {
namespace {

enum Fmt { MX = 0, NV = 1 };

constexpr int kFew = 64;  // assignments that a wave holds, one a lane

struct Args {
    const uint8_t *w13, *s13, *w2, *s2;
    const float *f13, *f2;
    const uint16_t *x;
    const int32_t *ids;
    const float *weights;
    uint16_t *out;
    int64_t xs, os;
    uint16_t *hi, *lo;  // h [assignments][inter], its bfloat16 and the rest
    float *y;           // [assignments][hidden]: results of W2, weighted (many assignments)
    const int32_t *list;  // more tokens: assignments by expert
    const int4 *slots;    // and each expert that has any: {its number, where its list begins, how many}; then {-1}
    int tokens, top, n, experts, hidden, inter;  // n: assignments
};

// 16 weight rows of k elements: where they start, the same in the whole wave. A lane's
// row (lane % 16) and block lie less than 2^32 bytes beyond.
struct Tile {
    const uint8_t *w, *s;
};
template <int F>
__device__ __forceinline__ Tile tile_of(const uint8_t *w, const uint8_t *s, int64_t row, int k) {
    return {w + row * (k / 2), s + row * (k / (F == MX ? 32 : 16))};
}
template <int F>
__device__ __forceinline__ const uint8_t *scales_end(const uint8_t *s, const Args &a, int rows, int k) {
    return s + (int64_t)a.experts * rows * (k / (F == MX ? 32 : 16));
}

// Eight elements, word i of a row's 32, as bfloat16, exact. scale: the 32's byte, or
// both bytes of NVFP4.
template <int F>
__device__ __forceinline__ bf16x8 expand(uint32_t c, uint32_t scale, int i) {
    u32x4 o;
    if constexpr (F == MX) {
        const float s = kv::e8m0_operand(scale);
        o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
        o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
        o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
        o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
    } else {
        const float s = e4m3fn_f32(i < 2 ? scale & 0xFFu : scale >> 8);
        const f32x2 a = e2m1x2_f32<0>(c), b = e2m1x2_f32<1>(c), d = e2m1x2_f32<2>(c), e = e2m1x2_f32<3>(c);
        o = u32x4{kv::pack2(a.x * s, a.y * s), kv::pack2(b.x * s, b.y * s), kv::pack2(d.x * s, d.y * s),
                  kv::pack2(e.x * s, e.y * s)};
    }
    return kv::as_bf16x8(o);
}

// h rounded to bfloat16, and what that leaves out, bfloat16 too: at most half of the first's
// last bit, 2^-8 of it, so that its own rounding is off by 2^-17 of h at most (with the first
// cut instead, 2^-16: twice as many outputs were rounded to another number than the nearest).
// Only where rounding would pass the largest number the first is cut: a finite h stays so.
__device__ __forceinline__ void split(float h, uint16_t &hi, uint16_t &lo) {
    const uint32_t b = __float_as_uint(h);
    if ((b & 0x7F800000u) == 0x7F800000u) {
        hi = bf16_bits_rne(h);
        lo = 0;
    } else {
        const uint16_t near = bf16_bits_rne(h);
        hi = (near & 0x7F80u) == 0x7F80u ? (uint16_t)(b >> 16) : near;
        lo = bf16_bits_rne(h - __uint_as_float((uint32_t)hi << 16));
    }
}

__device__ __forceinline__ float silu(float g) {
    return g * __builtin_amdgcn_rcpf(1.0f + kv::exp2_fast(-kv::kLog2e * g));
}

// Few assignments: the lanes that have lane `slot`'s expert (0 if it is none, or a lane
// before it has it too: then that one does the work).
__device__ __forceinline__ uint64_t same_expert(int id, bool valid, int slot, int &expert) {
    expert = __builtin_amdgcn_readlane(id, slot);
    const uint64_t m = __ballot(valid && id == expert);
    return m && __builtin_ctzll(m) == slot ? m : 0;
}
// The lane of the i-th bit of m.
__device__ __forceinline__ int nth_bit(uint64_t m, int i) {
    for (; i > 0; --i) m &= m - 1;
    return __builtin_ctzll(m);
}

// Loads go out here, in this order, not where they are used.
__device__ __forceinline__ void fix() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ---------------------------------------------------------------- scales
//
// A step of 256 elements wants 8 bytes of each row's scales (16 with NVFP4), from as many
// lines as the codes' 128: read with each step, they cost a third of the rate. So those of
// kSpan elements of 32 rows are copied into LDS first, 16 bytes a lane.
constexpr int kScaleBytes = 128;                 // of a row, that LDS holds
constexpr int kScalePitch = kScaleBytes + 16;    // so that 16 rows lie in as many banks
template <int F>
constexpr int kSpan = kScaleBytes * (F == MX ? 32 : 16);  // and their elements

// 16 bytes from s on, at any alignment; those from `end` on read as 0, and no byte there is touched
// (16 bytes lie before it). value() waits for them.
struct Bytes16 {
    u32x4 v;
    uint32_t beyond;  // bytes that the load lies before s

    __device__ __forceinline__ void load(const uint8_t *s, const uint8_t *end) {
        beyond = s > end - 16 ? (uint32_t)(s - (end - 16)) : 0;
        __builtin_memcpy(&v, s - beyond, 16);
    }
    __device__ __forceinline__ u32x4 value() const {
        u32x4 o = v;
        if (beyond & 8) o = u32x4{o.z, o.w, 0, 0};
        if (beyond & 4) o = u32x4{o.y, o.z, o.w, 0};
        return u32x4{__builtin_amdgcn_alignbyte(o.y, o.x, beyond), __builtin_amdgcn_alignbyte(o.z, o.y, beyond),
                     __builtin_amdgcn_alignbyte(o.w, o.z, beyond), __builtin_amdgcn_alignbyte(0, o.w, beyond)};
    }
};

// `count` blocks' scales, from block `first` on, of two tiles into LDS by 256 threads. end: of all scales.
// then(): called when the loads are on their way and before they are waited for.
template <int F, typename Then>
__device__ __forceinline__ void copy_scales(uint8_t *lds, const Tile (&tiles)[2], const uint8_t *end, uint32_t blocks,
                                            uint32_t first, uint32_t count, const Then &then) {
    constexpr int EACH = F == MX ? 1 : 2;  // bytes of a block
    const uint32_t row = threadIdx.x / 8, at = threadIdx.x % 8 * 16;
    Bytes16 v;
    v.load((row < 16 ? tiles[0].s : tiles[1].s) + (((row & 15) * blocks + first) * EACH + (at < count * EACH ? at : 0)), end);
    fix();
    then();
    *reinterpret_cast<u32x4 *>(lds + row * kScalePitch + at) = v.value();
}
// The scale, or both, of a block: row of 32, block of those that LDS has.
template <int F>
__device__ __forceinline__ uint32_t scale_of(const uint8_t *lds, int row, uint32_t block) {
    const uint8_t *s = lds + row * kScalePitch + block * (F == MX ? 1 : 2);
    if constexpr (F == MX) return *s;
    else return *reinterpret_cast<const uint16_t *>(s);
}

// ---------------------------------------------------------------- few tokens
//
// Each wave has its own part of k, all of whose loads it sends at once, and x (or h)
// lies in LDS as a whole: rows of `pitch` bytes, padded with zeros to whole pairs of steps.
// A step is 128 elements, 32 for each quarter of the lanes.
constexpr int kFewTokens = 8;

__host__ __device__ constexpr int few_pitch(int k) { return (k + 255) / 256 * 512 + 16; }

// Vectors of k bfloat16 values into LDS by a workgroup of WAVES waves, each 64 parts of 16 bytes of one
// vector at a time, AHEAD of those at once. from(r): where vector r lies. then(): as above.
template <int WAVES, int AHEAD, typename From, typename Then>
__device__ __forceinline__ void stage(uint8_t *lds, int rows, int k, const From &from, const Then &then) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t each = (k + 255) / 256 * 32, turns = (each + 63) / 64, total = rows * turns;
    const uint32_t inverse = turns > 1 ? 0xFFFFFFFFu / turns + 1 : 0;  // i / turns: i < 2^13
    const int pitch = few_pitch(k);
    const auto row_of = [&](uint32_t i) { return turns > 1 ? __umulhi(i, inverse) : i; };
    for (uint32_t i0 = wave;; i0 += WAVES * AHEAD) {
        u32x4 v[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const uint32_t i = min(i0 + u * WAVES, total - 1), r = row_of(i), at = (i - r * turns) * 64 + lane;
            const bool in = (int)at * 8 < k;
            v[u] = ld16(from((int)r) + (in ? at * 8 : 0));
            if (!in) v[u] = u32x4{0, 0, 0, 0};
        }
        if (i0 == (uint32_t)wave) {
            fix();
            then();
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const uint32_t i = i0 + u * WAVES, r = row_of(i), at = (i - r * turns) * 64 + lane;
            if (i < total && at < each) *reinterpret_cast<u32x4 *>(lds + r * pitch + at * 16) = v[u];
        }
        if (i0 + WAVES * AHEAD >= total) break;
    }
}

// COUNT pairs of steps from `first`, `every` apart, of a row tile. In pairs, since a
// row's two 64-byte halves of a line go through the first cache together then.
template <int F, int COUNT>
struct Batch {
    u32x4 codes[COUNT][2];
    uint32_t scale[COUNT][2];

    __device__ __forceinline__ void load(const Tile &tile, uint32_t blocks, uint32_t first, uint32_t every) {
        const uint32_t lane = threadIdx.x & 63, row = (lane & 15) * blocks;
#pragma unroll
        for (int u = 0; u < COUNT; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // beyond the row: its last block, and h is 0 there or not looked at
                const uint32_t at = row + min(8 * (first + u * every) + 4 * h + (lane >> 4), blocks - 1);
                codes[u][h] = ld16(tile.w + at * 16);
                if constexpr (F == MX) scale[u][h] = tile.s[at];
                else scale[u][h] = *reinterpret_cast<const uint16_t *>(tile.s + 2 * at);
            }
    }
    // Pairs below `pairs`. x: this lane's column in LDS, at its quarter
    __device__ __forceinline__ void multiply(const uint8_t *x, int pairs, int first, int every, f32x4 &acc) const {
#pragma unroll
        for (int u = 0; u < COUNT; ++u) {
            const int d = first + u * every;
            if (d >= pairs) break;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 v = kv::as_bf16x8(ld16(x + d * 512 + h * 256 + 16 * j));
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(expand<F>(codes[u][h][j], scale[u][h], j), v, acc, 0, 0, 0);
                }
        }
    }
};

// A workgroup has 16 gate and 16 up rows; its four waves split the pairs of steps among them and join
// their sums in LDS. What LDS has to have before the first product is loaded first, and the codes
// right after it, all of a span's: they then arrive while the first are multiplied.
constexpr int kGateWaves = 4;

// acc += a wave's part of a span, TURNS pairs of steps or fewer. x: this lane's column in LDS, at its quarter
template <int F, int TURNS, typename Stage>
__device__ __forceinline__ void gate_up_span(uint8_t *scales, const Tile (&tiles)[2], const uint8_t *end, uint32_t blocks, uint32_t start,
                                             uint32_t here, const uint8_t *x, const Stage &stage_x, f32x4 (&acc)[2]) {
    const uint32_t lane = threadIdx.x & 63, row = lane & 15, quarter = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), pairs = (here + 7) / 8;
    u32x4 p[TURNS][2][2];
    copy_scales<F>(scales, tiles, end, blocks, start, here, [&] {
        stage_x([&] {
#pragma unroll
            for (int u = 0; u < TURNS; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        p[u][h][i] = ld16(tiles[i].w + (row * blocks + start +
                                                        min(8 * (wave + u * kGateWaves) + 4 * h + quarter, here - 1)) * 16);
            fix();
        });
    });
    lds_barrier();
#pragma unroll
    for (int u = 0; u < TURNS; ++u) {
        const int d = wave + u * kGateWaves;
        if (d >= pairs) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t scale[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) scale[i] = scale_of<F>(scales, i * 16 + row, min(8 * d + 4 * h + quarter, here - 1));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 v = kv::as_bf16x8(ld16(x + d * 512 + h * 256 + 16 * j));
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(expand<F>(p[u][h][i][j], scale[i], j), v, acc[i], 0, 0, 0);
            }
        }
    }
}

template <int F>
__global__ __launch_bounds__(kGateWaves * 64, 3) void k_gate_up_few(Args a, int slots) {
    extern __shared__ __attribute__((aligned(16))) uint8_t xs[];
    __shared__ __attribute__((aligned(16))) uint8_t scales[32 * kScalePitch];
    __shared__ __attribute__((aligned(16))) float joined[kGateWaves][2][kFewTokens][16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row = lane & 15;
    const uint32_t quarter = lane >> 4;
    const int tile = blockIdx.x;
    const int id = lane < a.n ? a.ids[lane] : -1;
    int expert;
    const uint64_t m = same_expert(id, (uint32_t)id < (uint32_t)a.experts, blockIdx.y, expert);
    if (!m) return;
    const int n = __popcll(m), pitch = few_pitch(a.hidden);
    const uint32_t blocks = a.hidden / 32;
    const int64_t first = (int64_t)expert * 2 * a.inter + tile * 16;
    const Tile tiles[2] = {tile_of<F>(a.w13, a.s13, first, a.hidden), tile_of<F>(a.w13, a.s13, first + a.inter, a.hidden)};
    const uint8_t *const end = scales_end<F>(a.s13, a, 2 * a.inter, a.hidden);
    for (int g = 0; g < n; g += slots) {
        const int count = min(slots, n - g);
        f32x4 acc[2] = {};
        for (uint32_t start = 0; start < blocks; start += kSpan<F> / 32) {
            const uint32_t here = min(blocks - start, (uint32_t)kSpan<F> / 32);
            const uint8_t *x = xs + min(row, count - 1) * pitch + (start + quarter) * 64;
            const auto stage_x = [&](const auto &then) {
                if (start == 0)
                    stage<kGateWaves, 2>(
                        xs, count, a.hidden,
                        [&](int c) { return a.x + (int64_t)(nth_bit(m, g + c) / a.top) * a.xs; }, then);
                else then();
            };
            // Half of the loads where half are enough: the others would ask for the last block again (rows of 2048:
            // 9.9 us, else 11.6).
            constexpr int kMost = kSpan<F> / 256 / kGateWaves;
            if (here <= 16 * kGateWaves / 2 * (kMost / 2))
                gate_up_span<F, kMost / 2>(scales, tiles, end, blocks, start, here, x, stage_x, acc);
            else gate_up_span<F, kMost>(scales, tiles, end, blocks, start, here, x, stage_x, acc);
            if (start + kSpan<F> / 32 < blocks) __syncthreads();  // the scales are read
        }
        if (row < count)
#pragma unroll
            for (int i = 0; i < 2; ++i) *reinterpret_cast<f32x4 *>(&joined[wave][i][row][quarter * 4]) = acc[i];
        __syncthreads();
        const float f = F == NV ? a.f13[expert] : 1.0f;
        if ((int)threadIdx.x < count * 16) {
            const int c = threadIdx.x / 16, r = threadIdx.x % 16;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int j = 0; j < kGateWaves; ++j) gate += joined[j][0][c][r], up += joined[j][1][c][r];
            const int64_t to = (int64_t)nth_bit(m, g + c) * a.inter + tile * 16 + r;
            split(silu(gate * f) * (up * f), a.hi[to], a.lo[to]);
        }
        __syncthreads();
    }
}

// 16 output rows of all assignments. An item is an expert and a part of k (so that the
// waves have work where experts are fewer); its h lies in LDS, put there by the wave that
// needs it. Columns 0 .. 7 are the upper halves of the expert's h, 8 .. 15 the rests. An
// item's results, weighted, go to LDS, one place for each (part, assignment), and are
// added in a fixed order.
constexpr int kDownWaves = 16, kDownBatch = 3, kPlaces = 128;

template <int F>
__global__ __launch_bounds__(kDownWaves * 64) void k_down_few(Args a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t hs[];
    __shared__ __attribute__((aligned(16))) float part[kPlaces][16];
    __shared__ float factor[kFew];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row = lane & 15,
              quarter = lane >> 4;
    const int id = lane < a.n ? a.ids[lane] : -1;
    const bool valid = (uint32_t)id < (uint32_t)a.experts;
    const float weight = lane < a.n ? a.weights[lane] : 0.0f;  // lane: an assignment
    const int blocks = a.inter / 32, pairs = (blocks + 7) / 8, pitch = few_pitch(a.inter);
    int before = kFew;  // the first lane with this one's expert; a leader is its own
    for (int i0 = (a.n - 1) / 8 * 8; i0 >= 0; i0 -= 8)
#pragma unroll
        for (int i = 7; i >= 0; --i)
            if (__builtin_amdgcn_readlane(id, i0 + i) == id) before = i0 + i;
    const uint64_t leaders = __ballot(valid && before == lane);
    const int found = __popcll(leaders);
    int parts = 1;
    if (found > 0) parts = max(1, min(min(kDownWaves / found, kPlaces / a.n), pairs));
    const int items = found * parts;
    struct Item {
        uint64_t m;  // its assignments
        int p;       // its part: pairs p, p + parts, ...
        Tile tile;
        u32x4 h[kDownBatch];  // of the first assignment
        Batch<F, kDownBatch> batch;
    };
    // Pairs t, t + parts, ... of an assignment's h: lanes 0 .. 31 the upper halves, the others the rests.
    const auto load_h = [&](u32x4 (&h)[kDownBatch], int at, int t) {
        const uint16_t *from = (lane < 32 ? a.hi : a.lo) + (int64_t)at * a.inter;
#pragma unroll
        for (int u = 0; u < kDownBatch; ++u) {
            const int k = (t + u * parts) * 256 + (lane & 31) * 8;
            h[u] = ld16(from + (k < a.inter ? k : 0));
            if (k >= a.inter) h[u] = u32x4{0, 0, 0, 0};
        }
    };
    const auto store_h = [&](const u32x4 (&h)[kDownBatch], int at, int t) {
#pragma unroll
        for (int u = 0; u < kDownBatch; ++u)
            if (t + u * parts < pairs)
                *reinterpret_cast<u32x4 *>(hs + (2 * at + (lane >> 5)) * pitch + (t + u * parts) * 512 + (lane & 31) * 16) = h[u];
    };
    const auto begin = [&](Item &it, int item) {
        int expert;
        it.m = same_expert(id, valid, nth_bit(leaders, item % found), expert);
        it.p = item / found;
        it.tile = tile_of<F>(a.w2, a.s2, (int64_t)expert * a.hidden + blockIdx.x * 16, a.inter);
        load_h(it.h, nth_bit(it.m, 0), it.p);
        it.batch.load(it.tile, blocks, it.p, parts);
        fix();
    };
    Item it;
    if (wave < items) begin(it, wave);
    if (wave == 0) factor[lane] = valid ? weight * (F == NV ? a.f2[id] : 1.0f) : 0.0f;
    for (int item = wave; item < items; item += kDownWaves) {
        const int n = __popcll(it.m);
        Item next;
        if (item + kDownWaves < items) begin(next, item + kDownWaves);
        for (int g = 0; g < n; g += 8) {
            const int at = nth_bit(it.m, min(g + (row & 7), n - 1));
            const uint8_t *x = hs + (2 * at + (row >> 3)) * pitch + quarter * 64;
            f32x4 acc = {};
            for (int t = it.p; t < pairs; t += parts * kDownBatch) {
                if (t != it.p || g) it.batch.load(it.tile, blocks, t, parts);
                if (g == 0)
                    for (int c = 0; c < n; ++c) {
                        if (t != it.p || c) load_h(it.h, nth_bit(it.m, c), t);
                        store_h(it.h, nth_bit(it.m, c), t);
                    }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                it.batch.multiply(x, pairs, t, parts, acc);
            }
            f32x4 v = acc;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += dpp_f32<0x128>(v[i]);  // row_ror:8: the rest's column
            if (row < 8 && g + row < n) *reinterpret_cast<f32x4 *>(&part[it.p * a.n + at][quarter * 4]) = v;
        }
        if (item + kDownWaves < items) it = next;
    }
    __syncthreads();
    const uint64_t all = __ballot(valid);
    for (int i = threadIdx.x; i < a.tokens * 16; i += kDownWaves * 64) {
        const int t = i / 16, r = i % 16;
        float v = 0.0f;
        for (int j0 = 0; j0 < a.top; j0 += 8) {
            float y[8] = {};
            for (int p = 0; p < parts; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] += part[p * a.n + t * a.top + min(j0 + j, a.top - 1)][r];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = t * a.top + min(j0 + j, a.top - 1);
                if (j0 + j < a.top && all >> at & 1) v += y[j] * factor[at];
            }
        }
        a.out[t * a.os + blockIdx.x * 16 + r] = bf16_bits_rne(v);
    }
}

// ---------------------------------------------------------------- more tokens
//
// A workgroup's waves have 16 gate and 16 up rows (or 32 output rows) each, over all
// of k, and the same columns; then the next such rows of the same expert, `turns` times.
// All its pieces (256 elements of k) are one sequence: the loads of one turn's first
// pieces go out before the last turn's results are written, so that the start, five loads one
// after the other, is paid once.
//
// Columns come through LDS, a piece at a time, two in turn; they are loaded into registers
// two pieces ahead, so that the barrier between two pieces waits for no load that is younger
// than the weights it is multiplied with. Weights are loaded one piece ahead, a line at a
// time (its two halves one after the other: apart, each would ask the second cache for it);
// scales as above, but 32 bytes of each row at a time.
constexpr int kWaves = 8, kTiles = 4;  // tiles: of 16 columns, at most at a time
constexpr int kScaleTurn = 32;         // bytes of a row's scales at a time
struct Shared {
    u32x4 x[2][kTiles][32][16];
    u32x4 scales[kWaves][32][kScaleTurn / 16 + 1];
};

struct Pair {
    Tile tile[2];
};

// For each turn, done(turn, acc): acc[i][m] = 16 rows x 16 columns of (row tile i, columns' tile
// m). rows(turn): a wave's row tiles. column(m, c): where column c of tile m lies. end: of all
// scales.
//
// In LDS the columns' 16-byte parts lie part by part, a tile's 16 columns side by side
// in the order column ^ part: writes (32 parts of a column) and reads (16 columns of a
// part) both go through all banks.
template <int F, int XT, typename R, typename C, typename D>
__device__ __forceinline__ void stream(Shared &lds, int turns, const R &rows, const uint8_t *end, const C &column, int k,
                                       const D &done) {
    constexpr int EACH = F == MX ? 1 : 2, EVERY = kScaleTurn / EACH / 8;  // bytes of a block; pieces that 32 bytes last
    const uint32_t lane = threadIdx.x & 63, row = lane & 15, quarter = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t blocks = k / 32, pairs = (blocks + 7) / 8;
    // this thread's part of a piece, of a column of each tile
    const int part = threadIdx.x & 31, c = threadIdx.x >> 5;
    const uint16_t *x[XT];
#pragma unroll
    for (int i = 0; i < XT; ++i) x[i] = column(i, c);
    u32x4 xr[2][XT], p[2][2][2];
    Bytes16 sc;
    const auto load_x = [&](u32x4 (&v)[XT], uint32_t d) {
        const bool in = d * 256 + part * 8 < (uint32_t)k;
#pragma unroll
        for (int i = 0; i < XT; ++i) {
            v[i] = ld16(x[i] + (in ? d * 256 + part * 8 : 0));
            if (!in) v[i] = u32x4{0, 0, 0, 0};
        }
        fix();
    };
    const auto store_x = [&](const u32x4 (&v)[XT], int buf) {
#pragma unroll
        for (int i = 0; i < XT; ++i) lds.x[buf][i][part][c ^ (part & 15)] = v[i];
    };
    const auto load_w = [&](u32x4 (&q)[2][2], int turn, uint32_t d) {
        const Pair t = rows(turn);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[h][i] = ld16(t.tile[i].w + (row * blocks + min(8 * d + 4 * h + quarter, blocks - 1)) * 16);
        fix();
    };
    static_assert(kScaleTurn == 32, "16 bytes a lane, of 32 rows");
    const auto load_s = [&](int turn, uint32_t d) {  // for pieces d, d + 1, ... d + EVERY - 1
        const Pair t = rows(turn);
        const uint32_t at = d * 8 * EACH + (lane & 1) * 16;
        sc.load((lane < 32 ? t.tile[0].s : t.tile[1].s) + ((lane / 2 & 15) * blocks * EACH + (at < blocks * EACH ? at : 0)), end);
        fix();
    };
    const auto store_s = [&] { lds.scales[wave][lane / 2][lane & 1] = sc.value(); };
    uint32_t scale[2][2][2];  // [piece % 2][half][tile]
    const auto read_s = [&](uint32_t (&v)[2][2], uint32_t d) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *at = reinterpret_cast<const uint8_t *>(lds.scales[wave][i * 16 + row]) +
                                    (min(8 * d + 4 * h + quarter, blocks - 1) - d / EVERY * EVERY * 8) * EACH;
                if constexpr (F == MX) v[h][i] = *at;
                else v[h][i] = *reinterpret_cast<const uint16_t *>(at);
            }
    };
    const auto next = [&](int &turn, uint32_t &d) {  // the piece after, or the same where there is none
        if (d + 1 < pairs) ++d;
        else if (turn + 1 < turns) ++turn, d = 0;
    };
    int turn = 0, turn_w = 0;
    uint32_t d = 0, d_w = 0, d_x = 0;
    int turn_x = 0;
    load_s(0, 0);
    load_w(p[0], 0, 0);
    load_x(xr[0], 0);
    next(turn_x, d_x);
    load_x(xr[1], d_x);
    next(turn_w, d_w);
    store_s();
    read_s(scale[0], 0);
    store_x(xr[0], 0);
    lds_barrier();
    f32x4 acc[2][XT] = {};
    for (;;) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const bool first = d % EVERY == 0;
            if (first) {  // the next 32 bytes' turn
                const bool more = d + EVERY < pairs;
                load_s(more ? turn : min(turn + 1, turns - 1), more ? d + EVERY : 0);
            }
            next(turn_x, d_x);
            load_x(xr[u], d_x);
            load_w(p[u ^ 1], turn_w, d_w);
            next(turn_w, d_w);
            // Groups of steps with four column tiles' operands: a group's come from LDS while the one before is multiplied.
            constexpr int GROUP = 4 / XT;
            bf16x8 v[2][GROUP][XT];
            const auto read_x = [&](int g) {
#pragma unroll
                for (int q = 0; q < GROUP; ++q)
#pragma unroll
                    for (int m = 0; m < XT; ++m) {
                        const int step = g * GROUP + q, at = (step / 4 * 4 + quarter) * 4 + step % 4;
                        v[g & 1][q][m] = kv::as_bf16x8(lds.x[u][m][at][row ^ (at & 15)]);
                    }
            };
            read_x(0);
#pragma unroll
            for (int g = 0; g < 8 / GROUP; ++g) {
                __builtin_amdgcn_sched_barrier(0);
                if (g + 1 < 8 / GROUP) read_x(g + 1);
#pragma unroll
                for (int q = 0; q < GROUP; ++q) {
                    const int step = g * GROUP + q;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bf16x8 e = expand<F>(p[u][step / 4][i][step % 4], scale[u][step / 4][i], step % 4);
#pragma unroll
                        for (int m = 0; m < XT; ++m)
                            acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e, v[g & 1][q][m], acc[i][m], 0, 0, 0);
                    }
                }
            }
            fix();
            if (d % EVERY == EVERY - 1 || d + 1 == pairs) store_s();
            if (d + 1 == pairs) {
                done(turn, acc);
                if (turn + 1 == turns) return;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int m = 0; m < XT; ++m) acc[i][m] = f32x4{0, 0, 0, 0};
            }
            next(turn, d);
            read_s(scale[u ^ 1], d);
            store_x(xr[u ^ 1], u ^ 1);
            lds_barrier();
        }
    }
}

template <int F, int XT>
__device__ __forceinline__ void gate_up(const Args &a, Shared &lds, int group, int turns, int expert, int n, const int *list) {
    const int lane = threadIdx.x & 63, row = lane & 15, quarter = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), units = a.inter / 16;
    const auto rows = [&](int turn) {
        const int64_t first = (int64_t)expert * 2 * a.inter + min((group + turn) * kWaves + wave, units - 1) * 16;
        return Pair{{tile_of<F>(a.w13, a.s13, first, a.hidden), tile_of<F>(a.w13, a.s13, first + a.inter, a.hidden)}};
    };
    const auto column = [&](int m, int c) { return a.x + (int64_t)(list[min(16 * m + c, n - 1)] / a.top) * a.xs; };
    const float f = F == NV ? a.f13[expert] : 1.0f;
    int to[XT];
#pragma unroll
    for (int m = 0; m < XT; ++m) to[m] = list[min(16 * m + row, n - 1)];
    const auto done = [&](int turn, const f32x4 (&acc)[2][XT]) {
        const int unit = (group + turn) * kWaves + wave;
#pragma unroll
        for (int m = 0; m < XT; ++m) {
            if (unit >= units || 16 * m + row >= n) continue;
            uint16_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split(silu(acc[0][m][i] * f) * (acc[1][m][i] * f), hi[i], lo[i]);
            const int64_t at = (int64_t)to[m] * a.inter + unit * 16 + quarter * 4;
            *reinterpret_cast<u32x2 *>(a.hi + at) = u32x2{hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16};
            *reinterpret_cast<u32x2 *>(a.lo + at) = u32x2{lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16};
        }
    };
    stream<F, XT>(lds, turns, rows, scales_end<F>(a.s13, a, 2 * a.inter, a.hidden), column, a.hidden, done);
}

// The columns are h's upper halves and its rests: eight of each in one tile, or the
// tiles of the one and then those of the other. Either way their sums are added at the end, so that
// no result depends on which assignments come together.
template <int F, int XT>
__device__ __forceinline__ void down(const Args &a, Shared &lds, int group, int turns, int expert, int n, const int *list) {
    const int lane = threadIdx.x & 63, row = lane & 15, quarter = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), units = a.hidden / 32;
    const auto rows = [&](int turn) {
        const int64_t first = (int64_t)expert * a.hidden + min((group + turn) * kWaves + wave, units - 1) * 32;
        return Pair{{tile_of<F>(a.w2, a.s2, first, a.inter), tile_of<F>(a.w2, a.s2, first + 16, a.inter)}};
    };
    const auto column = [&](int m, int c) {
        const int at = 16 * m + c, half = 8 * XT;
        return (at < half ? a.hi : a.lo) + (int64_t)list[min(at % half, n - 1)] * a.inter;
    };
    constexpr int OUT = XT > 1 ? XT / 2 : 1;
    int to[OUT];
    float weight[OUT];
#pragma unroll
    for (int m = 0; m < OUT; ++m) {
        to[m] = list[min(16 * m + row, n - 1)];
        weight[m] = a.weights[to[m]] * (F == NV ? a.f2[expert] : 1.0f);
    }
    const auto done = [&](int turn, const f32x4 (&acc)[2][XT]) {
        const int unit = (group + turn) * kWaves + wave;
#pragma unroll
        for (int m = 0; m < OUT; ++m) {
            f32x4 v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    v[i][r] = acc[i][m][r] + (XT > 1 ? acc[i][(m + OUT) % XT][r] : dpp_f32<0x128>(acc[i][m][r]));  // row_ror:8
            if (unit >= units || 16 * m + row >= n || (XT == 1 && row >= 8)) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<f32x4 *>(a.y + (int64_t)to[m] * a.hidden + unit * 32 + i * 16 + quarter * 4) =
                    v[i] * weight[m];
        }
    };
    stream<F, XT>(lds, turns, rows, scales_end<F>(a.s2, a, a.hidden, a.inter), column, a.inter, done);
}

template <int F, bool DOWN>
__global__ __launch_bounds__(kWaves * 64) void k_stream(Args a, int turns) {
    __shared__ Shared lds;
    const int4 slot = a.slots[blockIdx.y];
    const int expert = slot.x, group = blockIdx.x * turns;
    if (expert < 0) return;
    turns = min(turns, (a.inter / 16 * !DOWN + a.hidden / 32 * DOWN + kWaves - 1) / kWaves - group);
    const int *list = a.list + slot.y;
    int n = slot.z;
    constexpr int EACH = DOWN ? 8 : 16;  // assignments that a tile of columns holds
    for (;;) {
        const int now = min(n, EACH * kTiles);
        if constexpr (DOWN) {
            if (now <= EACH) down<F, 1>(a, lds, group, turns, expert, now, list);
            else if (now <= 2 * EACH) down<F, 2>(a, lds, group, turns, expert, now, list);
            else down<F, 4>(a, lds, group, turns, expert, now, list);
        } else {
            if (now <= EACH) gate_up<F, 1>(a, lds, group, turns, expert, now, list);
            else if (now <= 2 * EACH) gate_up<F, 2>(a, lds, group, turns, expert, now, list);
            else gate_up<F, 4>(a, lds, group, turns, expert, now, list);
        }
        n -= EACH * kTiles, list += EACH * kTiles;
        if (n <= 0) return;
        lds_barrier();
    }
}

// out = the sum of a token's weighted results, in the order of its experts.
__global__ __launch_bounds__(256) void k_add(Args a) {
    const int64_t pieces = (int64_t)a.tokens * (a.hidden / 8);
    const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (p >= pieces) return;
    const int t = (int)(p / (a.hidden / 8)), i = (int)(p - (int64_t)t * (a.hidden / 8)) * 8;
    f32x4 sum[2] = {};
    for (int j0 = 0; j0 < a.top; j0 += 4) {  // four at a time: one after another they are latency alone
        f32x4 y[4][2];
        bool in[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = t * a.top + min(j0 + j, a.top - 1);
            in[j] = j0 + j < a.top && (uint32_t)a.ids[at] < (uint32_t)a.experts;
            const f32x4 *from = reinterpret_cast<const f32x4 *>(a.y + (int64_t)at * a.hidden + i);
            y[j][0] = from[0], y[j][1] = from[1];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (in[j]) sum[0] += y[j][0], sum[1] += y[j][1];
    }
    *reinterpret_cast<u32x4 *>(a.out + t * a.os + i) = u32x4{kv::pack2(sum[0].x, sum[0].y), kv::pack2(sum[0].z, sum[0].w),
                                                             kv::pack2(sum[1].x, sum[1].y), kv::pack2(sum[1].z, sum[1].w)};
}

// Many assignments: lists by expert, and the experts that have any (then -1). One
// workgroup. The order within an expert's list is left open: no result depends on it.
constexpr int kListThreads = 1024;
__global__ __launch_bounds__(kListThreads) void k_lists(Args a, int32_t *list, int4 *slots) {
    __shared__ int count[1024], at[1024];
    __shared__ int64_t scan[kListThreads / 64 + 1];
    const int e = threadIdx.x;
    count[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kListThreads) {
        const uint32_t id = (uint32_t)a.ids[i];
        if (id < (uint32_t)a.experts) atomicAdd(&count[id], 1);
    }
    __syncthreads();
    const int mine = count[e];
    int64_t total;
    // both sums at once: assignments below, experts with any above
    const int64_t before = kv::block_scan<kListThreads>((int64_t)mine | (int64_t)(mine > 0) << 32, scan, total);
    at[e] = (int)(uint32_t)before;
    if (mine > 0) slots[before >> 32] = make_int4(e, (int)(uint32_t)before, mine, 0);
    if (e < min(a.n, a.experts) && e >= (int)(total >> 32)) slots[e] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kListThreads) {
        const uint32_t id = (uint32_t)a.ids[i];
        if (id < (uint32_t)a.experts) list[atomicAdd(&at[id], 1)] = i;
    }
}

// The form for few tokens, where x and h fit LDS: both products of one token (8 of 64 experts, 4096 x 1536) take 23 us, 44
// in the other form with its lists and sums; of two (96 KiB of h) 39 and 47; of 7 tokens (4 of 32, 1120 x 736, nvfp4) 22 and
// 29; of one (2 of 8, 4096 x 14336, 112 KiB) 52 and 107. The bound on h lies below what the kernel's own 8.5 KiB leave of a
// workgroup's 160, and short of where the forms cross: from 128 KiB on this one would be ahead by 2 % (two tokens, inter
// 2048, 128.5 KiB: 51.8 and 52.7) to a fifth (three, inter 1536, 145 KiB: 50 and 65).
constexpr int kFewLds = 128 << 10;
bool is_few(const qbn_moe_weights &e, int64_t tokens, int top) {
    return tokens <= kFewTokens && tokens * top <= kFew && few_pitch(e.hidden) <= kFewLds &&
           tokens * top * 2 * few_pitch(e.inter) <= kFewLds;
}

struct Layout {  // of the workspace, in bytes
    int64_t hi, lo, y, slots, list, end;
};
Layout layout_of(const qbn_moe_weights &e, int64_t tokens, int top) {
    const int64_t n = (tokens < QBN_MOE_PORTION ? tokens : QBN_MOE_PORTION) * top;
    const bool few = is_few(e, tokens, top);
    Layout l;
    l.hi = 0;
    l.lo = l.hi + n * e.inter * 2;
    l.y = l.lo + n * e.inter * 2;
    l.slots = l.y + (few ? 0 : n * e.hidden * 4);
    l.list = l.slots + (few ? 0 : e.experts * (int64_t)sizeof(int4));
    l.end = l.list + (few ? 0 : n * 4);
    return l;
}

// Workgroups that a kernel of streams should have at least, two for a compute unit, before each takes more than one
// group of rows: with 256 the last are waited for (64 tokens of 64 experts, first product: 53 us, with 512 47), with as
// many as there are groups each pays its start (256 tokens of 128 experts, second product: 135 us, with 512 127). Layers of few
// or narrow experts have fewer groups than that in all, and compute units without work (12 tokens, 4 experts of 4096 x
// 1024: both products, lists and sums 35 us for 27 MB).
constexpr int kEnough = 512;

template <int F>
hipError_t launch(const Args &a, bool few, int32_t *list, int4 *where, hipStream_t s) {
    if (few) {
        const int pitch = few_pitch(a.hidden), slots = a.tokens < kFewLds / pitch ? a.tokens : kFewLds / pitch;
        const dim3 grid(a.inter / 16, a.n);
        k_gate_up_few<F><<<grid, kGateWaves * 64, slots * pitch, s>>>(a, slots);
        k_down_few<F><<<a.hidden / 16, kDownWaves * 64, 2 * a.n * few_pitch(a.inter), s>>>(a);
    } else {
        const int slots = a.n < a.experts ? a.n : a.experts;
        k_lists<<<1, kListThreads, 0, s>>>(a, list, where);
        const auto turns_of = [&](int groups) {
            const int t = std::max(1, std::min(groups, groups * slots / kEnough)), n = (groups + t - 1) / t;
            return (groups + n - 1) / n;
        };
        const int up = (a.inter / 16 + kWaves - 1) / kWaves, out = (a.hidden / 32 + kWaves - 1) / kWaves;
        const int tu = turns_of(up), td = turns_of(out);
        k_stream<F, false><<<dim3((up + tu - 1) / tu, slots), kWaves * 64, 0, s>>>(a, tu);
        k_stream<F, true><<<dim3((out + td - 1) / td, slots), kWaves * 64, 0, s>>>(a, td);
        const int64_t blocks = ((int64_t)a.tokens * (a.hidden / 8) + 255) / 256;
        k_add<<<(unsigned)blocks, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

int64_t moe_experts_workspace(const qbn_moe_weights &e, int64_t tokens, int top_k) {
    return tokens > 0 ? layout_of(e, tokens, top_k).end : 0;
}

hipError_t launch_moe_experts(const qbn_moe_weights &e, int64_t tokens, int top_k, const void *x, int64_t x_stride,
                              const int32_t *ids, const float *weights, void *out, int64_t out_stride, void *ws,
                              hipStream_t s) {
    const Layout l = layout_of(e, tokens, top_k);
    uint8_t *b = (uint8_t *)ws;
    Args a = {};
    a.w13 = (const uint8_t *)e.w13, a.s13 = (const uint8_t *)e.w13_scales, a.f13 = e.w13_scale2;
    a.w2 = (const uint8_t *)e.w2, a.s2 = (const uint8_t *)e.w2_scales, a.f2 = e.w2_scale2;
    a.xs = x_stride, a.os = out_stride;
    a.top = top_k, a.experts = e.experts, a.hidden = e.hidden, a.inter = e.inter;
    a.hi = (uint16_t *)(b + l.hi), a.lo = (uint16_t *)(b + l.lo), a.y = (float *)(b + l.y);
    int32_t *list = (int32_t *)(b + l.list);
    int4 *slots = (int4 *)(b + l.slots);
    a.list = list, a.slots = slots;
    const bool few = is_few(e, tokens, top_k);  // of the whole call: the last portion's tokens are summed as the others'
    for (int64_t at = 0; at < tokens; at += QBN_MOE_PORTION) {
        a.tokens = (int)(tokens - at < QBN_MOE_PORTION ? tokens - at : QBN_MOE_PORTION), a.n = a.tokens * top_k;
        a.x = (const uint16_t *)x + at * x_stride, a.out = (uint16_t *)out + at * out_stride;
        a.ids = ids + at * top_k, a.weights = weights + at * top_k;
        const hipError_t st = e.format == QBN_MXFP4 ? launch<MX>(a, few, list, slots, s) : launch<NV>(a, few, list, slots, s);
        if (st != hipSuccess) return st;
    }
    return hipSuccess;
}

}  // namespace qbn
