// Attention of one new token per sequence over the paged key-value cache.
//
//   s_j = c q.k_j,  out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m)
//
// with c = scale log2 e and m a running reference of the maximum. Bound by
// the cache's bytes; what has to be kept up with them is the expansion of the
// elements to bf16 and their product with the (up to 16) query heads that
// share a key-value head.
//
// Layout of the work. A wave takes 32 tokens at a time and computes the
// TRANSPOSED scores K Q^T (16x16x32 bf16 MFMA: rows are tokens, columns query
// heads), because a lane then holds eight scores of one head, and, with the
// 32 rows of K fed in the order below, exactly the eight tokens that the lane
// has to supply as the right operand of V^T P^T. So the softmax weights never
// leave their lane: no LDS, no cross-lane moves. The reduction axes are free
// to be permuted, which is used twice: lane group g of K reads whole
// contiguous pieces of a token's head (16 bytes = one MX block of E2M1 at
// head_dim 128), and V's rows are assigned to lanes so that a lane's part of
// a token is contiguous; eight tokens of it are turned into matrix operands
// by v_perm in registers.
//
// The reference m is raised only when a score exceeds it by 2^8 (a wave-wide
// vote), so the usual tile needs no cross-lane maximum and no rescaling:
// the weights then stay below 2^8 and binary32 sums hold them.
//
// Splitting. The tiles of all (sequence, head group) pairs form one list that
// a fixed number of workgroups shares evenly, whatever the lengths; each
// workgroup finds its piece from the lengths (one scan). A pair that lies in
// one workgroup is written at once; the pieces of the others go through the
// workspace and a second kernel joins them in order.
#include "kv_device.h"
#include "kv_launch.h"

namespace qbn {
namespace {

using namespace kv;

constexpr int kUnit = 128;  // tokens per unit of work: 4 waves x 32

struct DecodeArgs {
    Cache c;
    Batch b;
    const __bf16 *q;
    int64_t qt, qh;
    __bf16 *out;
    float *lse;
    float *parts;  // slots of [16][D] sums, then [16] maxima and [16] sums of weights
    float scale;   // times log2 e
    int group, tiles, rows;  // query heads per key-value head, 16-row tiles of them, pairs per sequence
    int window, sinks, blocks, dim;
};

// Units of 128 tokens that a sequence's query sees: those of the sinks, then
// those of the window.
struct Span {
    int len, lo, first, sink_units, n;
    bool bad;
};

__device__ __forceinline__ Span span_of(const DecodeArgs &a, int len) {
    Span s;
    s.bad = len < 0 || (((int64_t)len + (1 << a.c.page_shift) - 1) >> a.c.page_shift) > a.b.row;
    s.len = s.bad ? 0 : len;
    s.lo = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
    s.first = s.lo / kUnit;
    s.sink_units = min((min(a.sinks, s.lo) + kUnit - 1) / kUnit, s.first);
    s.n = s.sink_units + (int)(((int64_t)s.len + kUnit - 1) / kUnit) - s.first;
    return s;
}

__device__ __forceinline__ int64_t per_block(const DecodeArgs &a, int64_t total) {
    const int64_t p = (total + a.blocks - 1) / a.blocks;
    return p < 2 ? 2 : p;
}

// A wave's 32 tokens as loaded: K rows, V rows and their scales.
template <int F, int D>
struct Tile {
    // K: a lane group's contiguous piece of E elements, NC pieces per row
    static constexpr int E = F == FP4 ? (D % 128 == 0 ? 32 : D % 64 == 0 ? 16 : 8) : F == FP8 ? (D % 64 == 0 ? 16 : 8) : 8;
    static constexpr int NC = D / (4 * E);
    static constexpr int KB = E * kBits<F> / 8, KW = KB / 4;
    // V: 16 lanes cover 128, 64 or 32 elements of a row
    static constexpr int N8 = D / 128, N4 = D % 128 / 64, N2 = D % 64 / 32, NS = N8 + N4 + N2;
    static constexpr int words(int w) { return w * kBits<F> / 32 > 0 ? w * kBits<F> / 32 : 1; }
    static constexpr int W8 = words(8), W4 = words(4), W2 = words(2);
    uint32_t k[2][NC * KW];
    uint32_t ks[F == BF16 ? 1 : 2][F == BF16 ? 1 : NC];
    uint32_t v[8][N8 * W8 + N4 * W4 + N2 * W2];
    u32x2 vs[F == BF16 ? 1 : NS];
};

template <int F, int D>
struct Decoder {
    using T = Tile<F, D>;
    const DecodeArgs &a;
    int lane, m, g, kv_head, b;
    Span sp;
    bool bad = false;

    __device__ __forceinline__ bool sees(int t) const { return t < sp.len && (t >= sp.lo || t < a.sinks); }

    // The page of tokens t .. t + 15 (t % 16 == 0): page 0 where none of them is seen.
    __device__ __forceinline__ int64_t page_of(int t) {
        const bool any = t < sp.len && (t + 15 >= sp.lo || t < a.sinks);
        if (!any) return 0;
        const int p = a.b.table[(int64_t)b * a.b.row_stride + (t >> a.c.page_shift)];
        if ((uint32_t)p >= (uint32_t)a.c.pages) {
            bad = true;
            return 0;
        }
        return p;
    }

    __device__ __forceinline__ void load(T &r, int t0) {
        const int ps = 1 << a.c.page_shift;
        const int64_t p0 = page_of(t0), p1 = page_of(t0 + 16);
        // K: rows 4g' + i of the first product are tokens 8g' + i, of the second 8g' + 4 + i
        {
            const int t = 8 * (m / 4) + m % 4;  // < 16 for m < 8
            const int64_t head = (m < 8 ? p0 : p1) * a.c.heads + kv_head;
            const int slot = (t0 + t) & (ps - 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *row = a.c.k + ((head * ps + slot + 4 * i) * D) * kBits<F> / 8;
#pragma unroll
                for (int c = 0; c < T::NC; ++c) load_words<T::KB>(row + (c * 4 + g) * T::KB, r.k[i] + c * T::KW);
                if constexpr (F != BF16) {
                    const uint8_t *sc = a.c.ks + head * (D / 32) * ps + slot + 4 * i;
#pragma unroll
                    for (int c = 0; c < T::NC; ++c) r.ks[i][c] = sc[(c * 4 + g) * T::E / 32 * ps];
                }
            }
        }
        {
            const int64_t head = (g < 2 ? p0 : p1) * a.c.heads + kv_head;
            const int slot = (t0 + 8 * g) & (ps - 1);
            const uint8_t *row = a.c.v + ((head * ps + slot) * D) * kBits<F> / 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint8_t *p = row + j * (D * kBits<F> / 8);
#pragma unroll
                for (int n = 0; n < T::N8; ++n) load_words<kBits<F>>(p + (n * 128 + m * 8) * kBits<F> / 8, r.v[j] + n * T::W8);
                if constexpr (T::N4 > 0)
                    load_words<4 * kBits<F> / 8>(p + (T::N8 * 128 + m * 4) * kBits<F> / 8, r.v[j] + T::N8 * T::W8);
                if constexpr (T::N2 > 0)
                    load_words<2 * kBits<F> / 8>(p + (T::N8 * 128 + T::N4 * 64 + m * 2) * kBits<F> / 8,
                                                 r.v[j] + T::N8 * T::W8 + T::N4 * T::W4);
            }
            if constexpr (F != BF16) {
                const uint8_t *sc = a.c.vs + head * (D / 32) * ps + slot;
#pragma unroll
                for (int n = 0; n < T::N8; ++n) r.vs[n] = ld8(sc + (n * 4 + m / 4) * ps);
                if constexpr (T::N4 > 0) r.vs[T::N8] = ld8(sc + (T::N8 * 4 + m / 8) * ps);
                if constexpr (T::N2 > 0) r.vs[T::N8 + T::N4] = ld8(sc + (T::N8 * 4 + T::N4 * 2) * ps);
            }
        }
    }

    // V of the tokens that the query does not see becomes 0: their weights are
    // 0, and 0 times what lies there must not be NaN.
    __device__ __forceinline__ void clear_unseen(T &r, int t0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool on = sees(t0 + 8 * g + j);
#pragma unroll
            for (uint32_t &w : r.v[j]) w = on ? w : 0u;
            if constexpr (F != BF16) {
                const uint32_t mask = 0xFFu << (8 * (j & 3));
#pragma unroll
                for (u32x2 &s : r.vs) {
                    if (j < 4) s.x = on ? s.x : (s.x & ~mask);
                    else s.y = on ? s.y : (s.y & ~mask);
                }
            }
        }
    }

    template <int W>
    __device__ __forceinline__ void add_segment(const T &r, int word, u32x2 vs, bf16x8 p, f32x4 *acc) {
        uint32_t c[8][W / 2];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float sc = F == BF16 ? 1.0f : e8m0_f32((j < 4 ? vs.x : vs.y) >> (8 * (j & 3)));
            expand<F, W>(r.v[j] + word, sc, c[j]);
        }
#pragma unroll
        for (int t = 0; t < W; ++t)
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(column8<W>(c, t)), p, acc[t], 0, 0, 0);
    }

    __device__ __forceinline__ void step(T &r, int t0, const bf16x8 *q, float &ref, float &sum, f32x4 *acc) {
        // whole tiles that every query head sees need no mask
        const bool whole = t0 + 31 < sp.len && (t0 >= sp.lo || t0 + 31 < a.sinks);
        f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < T::NC; ++c) {
                const float sc = F == BF16 ? 1.0f : e8m0_f32(r.ks[i][F == BF16 ? 0 : c]);
#pragma unroll
                for (int e = 0; e < T::E / 8; ++e) {
                    uint32_t o[4];
                    expand8<F>(r.k[i] + c * T::KW + e * (kBits<F> / 4), sc, o);
                    s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(u32x4{o[0], o[1], o[2], o[3]}),
                                                                   q[c * (T::E / 8) + e], s[i], 0, 0, 0);
                }
            }
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s[j / 4][j & 3] * a.scale;
        if (!whole) {
            clear_unseen(r, t0);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = sees(t0 + 8 * g + j) ? x[j] : kNegInf;
        }
        float top = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = __builtin_fmaxf(top, x[j]);
        if (__any(top > ref + 8.0f)) {
            top = __builtin_fmaxf(top, __shfl_xor(top, 16));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            const float now = __builtin_fmaxf(ref, top);
            const float f = now == ref ? 1.0f : exp2_fast(ref - now);
            ref = now;
            sum *= f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) acc[t] *= f;
        }
        const float base = ref == kNegInf ? 0.0f : ref;
        u32x4 p;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float p0 = exp2_fast(x[j] - base), p1 = exp2_fast(x[j + 1] - base);
            sum += p0 + p1;
            p[j / 2] = pack_bf16x2(p0, p1);
        }
        const bf16x8 pb = as_bf16x8(p);
#pragma unroll
        for (int n = 0; n < T::N8; ++n) add_segment<8>(r, n * T::W8, r.vs[F == BF16 ? 0 : n], pb, acc + 8 * n);
        if constexpr (T::N4 > 0)
            add_segment<4>(r, T::N8 * T::W8, r.vs[F == BF16 ? 0 : T::N8], pb, acc + 8 * T::N8);
        if constexpr (T::N2 > 0)
            add_segment<2>(r, T::N8 * T::W8 + T::N4 * T::W4, r.vs[F == BF16 ? 0 : T::N8 + T::N4], pb,
                           acc + 8 * T::N8 + 4 * T::N4);
    }

    __device__ __forceinline__ int unit_token(int u) const {
        return (u < sp.sink_units ? u : u - sp.sink_units + sp.first) * kUnit;
    }
};

template <int F, int D>
__global__ __launch_bounds__(256) void k_decode(DecodeArgs a) {
    using T = Tile<F, D>;
    constexpr int LD = D + 4;  // padded row: 16 heads' writes of one element land in different banks
    __shared__ float s_acc[4][16][LD];
    __shared__ float s_ref[4][16], s_sum[4][16];
    __shared__ int64_t s_scan[5];
    __shared__ int64_t s_start[2];  // sequence, units before it
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // ---- this workgroup's piece of the list of units
    int b, r, off;
    int64_t left;
    if (a.parts == nullptr) {  // one workgroup per pair
        b = blockIdx.x / a.rows;
        r = blockIdx.x % a.rows;
        off = 0;
        left = (int64_t)1 << 40;
    } else {
        const int each = (a.b.seqs + 255) / 256;
        int64_t mine = 0;
        for (int i = 0; i < each; ++i) {
            const int s = tid * each + i;
            if (s < a.b.seqs) mine += span_of(a, a.b.lens[s]).n;
        }
        int64_t total;
        int64_t before = block_scan<256>(mine, s_scan, total);
        const int64_t per = per_block(a, total * a.rows), start = blockIdx.x * per;
        if (start >= total * a.rows) return;
        if (before * a.rows <= start && start < (before + mine) * a.rows) {
            for (int i = 0; i < each; ++i) {
                const int s = tid * each + i;
                const int n = span_of(a, a.b.lens[s]).n;
                if (start < (before + n) * a.rows) {
                    s_start[0] = s;
                    s_start[1] = before;
                    break;
                }
                before += n;
            }
        }
        __syncthreads();
        b = (int)s_start[0];
        const int64_t rem = start - s_start[1] * a.rows;
        const int n = span_of(a, a.b.lens[b]).n;
        r = (int)(rem / n);
        off = (int)(rem % n);
        left = per;
    }

    while (left > 0 && b < a.b.seqs) {
        Decoder<F, D> w{a};
        w.lane = lane;
        w.m = lane & 15;
        w.g = lane >> 4;
        w.b = __builtin_amdgcn_readfirstlane(b);
        w.kv_head = __builtin_amdgcn_readfirstlane(r / a.tiles);
        w.sp = span_of(a, a.b.lens[w.b]);
        const int n = w.sp.n, u1 = (int)(off + left < n ? off + left : n);
        if (n > 0 || a.parts == nullptr) {
            const int h0 = r % a.tiles * 16, heads = min(16, a.group - h0);
            const int hq = w.kv_head * a.group + h0;  // first query head of the pair
            // Q as the right operand, in the element order of K's pieces
            bf16x8 q[D / 32];
#pragma unroll
            for (int s = 0; s < D / 32; ++s) {
                const int d = (s * 8 / T::E * 4 + w.g) * T::E + s * 8 % T::E;
                u32x4 t = {0, 0, 0, 0};
                if (w.m < heads) t = ld16(a.q + (int64_t)w.b * a.qt + (int64_t)(hq + w.m) * a.qh + d);
                q[s] = as_bf16x8(t);
            }
            f32x4 acc[D / 16];
#pragma unroll
            for (int t = 0; t < D / 16; ++t) acc[t] = f32x4{0, 0, 0, 0};
            float ref = kNegInf, sum = 0.0f;
            T cur, nxt;
            if (off < u1) w.load(cur, w.unit_token(off) + 32 * wave);
            for (int u = off; u < u1; u += 2) {
                if (u + 1 < u1) w.load(nxt, w.unit_token(u + 1) + 32 * wave);
                w.step(cur, w.unit_token(u) + 32 * wave, q, ref, sum, acc);
                if (u + 1 < u1) {
                    if (u + 2 < u1) w.load(cur, w.unit_token(u + 2) + 32 * wave);
                    w.step(nxt, w.unit_token(u + 1) + 32 * wave, q, ref, sum, acc);
                }
            }
            // ---- the four waves' sums meet in LDS
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (w.bad || w.sp.bad) sum = __builtin_nanf("");
            if (lane < 16) {
                s_ref[wave][lane] = ref;
                s_sum[wave][lane] = sum;
            }
            __syncthreads();
            {
                float top = s_ref[0][w.m];
#pragma unroll
                for (int i = 1; i < 4; ++i) top = __builtin_fmaxf(top, s_ref[i][w.m]);
                const float f = ref == top ? 1.0f : exp2_fast(ref - top);
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    constexpr int A8 = T::N8 * 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 4 * w.g + i;
                        const int d = t < A8 ? t / 8 * 128 + row * 8 + t % 8
                                             : t < A8 + 4 * T::N4 ? T::N8 * 128 + row * 4 + (t - A8)
                                                                  : T::N8 * 128 + T::N4 * 64 + row * 2 + (t - A8 - 4 * T::N4);
                        s_acc[wave][w.m][d] = acc[t][i] * f;
                    }
                }
            }
            __syncthreads();
            const bool all = off == 0 && u1 == n;
            const int64_t slot = (int64_t)blockIdx.x + (int64_t)w.b * a.rows + r;
            float *part = a.parts + slot * (16 * D + 32);
            for (int i = tid; i < heads * (D / 4); i += 256) {
                const int h = i / (D / 4), d = i % (D / 4) * 4;
                float top = s_ref[0][h];
#pragma unroll
                for (int k = 1; k < 4; ++k) top = __builtin_fmaxf(top, s_ref[k][h]);
                float total = 0.0f;
                f32x4 o = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float rk = s_ref[k][h];
                    total += s_sum[k][h] * (rk == top ? 1.0f : exp2_fast(rk - top));
                    o += *reinterpret_cast<const f32x4 *>(&s_acc[k][h][d]);
                }
                if (all) {
                    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
                    const int64_t row = (int64_t)w.b * a.rows / a.tiles * a.group + hq + h;
                    *reinterpret_cast<u32x2 *>(a.out + row * D + d) =
                        u32x2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
                    if (d == 0 && a.lse) a.lse[row] = total == 0.0f ? kNegInf : (top + __builtin_amdgcn_logf(total)) * kLn2;
                } else {
                    *reinterpret_cast<f32x4 *>(part + h * D + d) = o;
                    if (d == 0) {
                        part[16 * D + h] = top;
                        part[16 * D + 16 + h] = total;
                    }
                }
            }
            __syncthreads();  // before the next pair overwrites LDS
        }
        if (a.parts == nullptr) return;
        left -= u1 - off;
        off = 0;
        if (++r == a.rows) {
            r = 0;
            ++b;
        }
    }
}

// Joins the pieces of each pair, in order: a wave per (sequence, query head).
template <int D>
__global__ __launch_bounds__(256) void k_decode_join(DecodeArgs a) {
    __shared__ int64_t s_scan[5];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int quads = (a.group + 3) / 4;  // workgroups per key-value head: four query heads each
    const int kv_heads = a.rows / a.tiles;
    const int b = blockIdx.x / (kv_heads * quads), rest = blockIdx.x % (kv_heads * quads);
    const int kv_head = rest / quads, hg = rest % quads * 4 + wave;
    // units before this sequence, and of all
    int64_t mine = 0, all = 0;
    for (int s = tid; s < a.b.seqs; s += 256) {
        const int n = span_of(a, a.b.lens[s]).n;
        all += n;
        if (s < b) mine += n;
    }
    int64_t total, before;
    block_scan<256>(all, s_scan, total);
    block_scan<256>(mine, s_scan, before);
    const Span sp = span_of(a, a.b.lens[b]);
    if (hg >= a.group) return;
    const int64_t row = ((int64_t)b * kv_heads + kv_head) * a.group + hg;
    if (sp.n == 0) {
        const float none = sp.bad ? __builtin_nanf("") : 0.0f;
        for (int d = lane; d < D; d += 64) a.out[row * D + d] = (__bf16)none;
        if (lane == 0 && a.lse) a.lse[row] = sp.bad ? none : kNegInf;
        return;
    }
    const int64_t per = per_block(a, total * a.rows);
    const int r = kv_head * a.tiles + hg / 16;
    const int64_t u0 = before * a.rows + (int64_t)r * sp.n;
    const int64_t i0 = u0 / per, i1 = (u0 + sp.n - 1) / per;
    if (i0 == i1) return;  // written by its workgroup
    const float *part = a.parts + (i0 + (int64_t)b * a.rows + r) * (16 * D + 32);
    const int h = hg % 16, count = (int)(i1 - i0 + 1);
    float top = kNegInf;
    for (int i = lane; i < count; i += 64) top = __builtin_fmaxf(top, part[(int64_t)i * (16 * D + 32) + 16 * D + h]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
    constexpr int PER = (D + 63) / 64;
    float o[PER] = {}, sum = 0.0f;
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
        const float *p = part + (int64_t)i * (16 * D + 32);
        const float ri = p[16 * D + h];
        const float f = ri == top ? 1.0f : exp2_fast(ri - top);
        sum += f * p[16 * D + 16 + h];
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (D % 64 == 0 || e * 64 + lane < D) o[e] += f * p[h * D + e * 64 + lane];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < PER; ++e)
        if (D % 64 == 0 || e * 64 + lane < D) a.out[row * D + e * 64 + lane] = (__bf16)(o[e] * inv);
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.0f ? kNegInf : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// How the host cuts the work: the most units a sequence can have (from the
// table's width, the window and the sinks), and the number of workgroups.
struct Plan {
    int64_t units, pairs, blocks;
    int tiles;
};

Plan plan_of(const qbn_kv_cache &c, const qbn_kv_batch &b, int q_heads, int window, int sinks) {
    Plan p;
    p.tiles = (q_heads / c.heads + 15) / 16;
    p.pairs = b.seqs * c.heads * p.tiles;
    p.units = (b.row * c.page_size + kUnit - 1) / kUnit;
    if (window > 0) {
        const int64_t seen = (int64_t)window / kUnit + 2 + ((int64_t)sinks + kUnit - 1) / kUnit;
        if (seen < p.units) p.units = seen;
    }
    // Up to two units a pair: one workgroup each. More: 1024 workgroups, four
    // per compute unit, share the units.
    p.blocks = p.units <= 2 ? 0 : p.pairs * p.units / 2 < 1024 ? p.pairs * p.units / 2 + 1 : 1024;
    return p;
}

template <int F>
hipError_t launch(const DecodeArgs &a, int64_t grid, int64_t join, hipStream_t s) {
    const dim3 g((unsigned)grid), gj((unsigned)join);
#define QBN_KV_DIM(DD)                                            \
    case DD:                                                      \
        k_decode<F, DD><<<g, 256, 0, s>>>(a);                     \
        if (a.parts) k_decode_join<DD><<<gj, 256, 0, s>>>(a);     \
        break;
    switch (a.dim) {
        QBN_KV_DIM(64)
        QBN_KV_DIM(96)
        QBN_KV_DIM(128)
        QBN_KV_DIM(192)
        QBN_KV_DIM(256)
    }
#undef QBN_KV_DIM
    return hipGetLastError();
}

}  // namespace

int64_t kv_decode_workspace(const qbn_kv_cache &c, const qbn_kv_batch &b, int q_heads, int window, int sinks) {
    const Plan p = plan_of(c, b, q_heads, window, sinks);
    return p.blocks ? (p.blocks + p.pairs) * (16 * (int64_t)c.head_dim + 32) * 4 : 0;
}

hipError_t launch_kv_decode(const qbn_kv_cache &c, int64_t layer, const qbn_kv_batch &b, int q_heads, const KvRows &q,
                            float scale, int window, int sinks, void *out, float *lse, void *ws, hipStream_t s) {
    const Plan p = plan_of(c, b, q_heads, window, sinks);
    const int64_t elems = layer * c.pages * c.heads * c.page_size * c.head_dim;
    const int bits = c.format == QBN_KV_BF16 ? 16 : c.format == QBN_MXFP8 ? 8 : 4;
    DecodeArgs a;
    a.c = {(const uint8_t *)c.k + elems * bits / 8, (const uint8_t *)c.v + elems * bits / 8,
           (const uint8_t *)c.k_scales + elems / 32, (const uint8_t *)c.v_scales + elems / 32, c.heads,
           __builtin_ctz(c.page_size), (int)c.pages};
    a.b = {(int)b.seqs, (int)b.tokens, (int)b.row, b.row_stride, b.table, b.lens, nullptr};
    a.q = (const __bf16 *)q.p;
    a.qt = q.token_stride, a.qh = q.head_stride;
    a.out = (__bf16 *)out, a.lse = lse;
    a.parts = p.blocks ? (float *)ws : nullptr;
    a.scale = scale * kLog2e;
    a.group = q_heads / c.heads, a.tiles = p.tiles, a.rows = c.heads * p.tiles;
    a.window = window, a.sinks = sinks, a.blocks = (int)p.blocks, a.dim = c.head_dim;
    const int64_t grid = p.blocks ? p.blocks : p.pairs;
    const int64_t join = b.seqs * c.heads * ((a.group + 3) / 4);
    if (c.format == QBN_KV_BF16) return launch<BF16>(a, grid, join, s);
    return c.format == QBN_MXFP8 ? launch<FP8>(a, grid, join, s) : launch<FP4>(a, grid, join, s);
}

}  // namespace qbn
