// Causal attention of chunks of new tokens over the paged key-value cache,
// with a sliding window and sink tokens.
//
// The rows of a workgroup are (token, query head) pairs of one key-value head:
// heads that share K and V share the loads and the expansion to bf16, and a
// chunk of a few tokens still fills rows. K and V go through LDS in tiles of
// 64 tokens, two buffers, the next tile's bytes in registers while this one
// is computed. Both lie there as [token][head_dim], rows padded by 16 (K) and
// 32 bytes (V): K's matrix operand is 16 bytes of a row, V's is read column
// by column with the transposing LDS load, four tokens at a time.
//
// The products are transposed: S^T = K Q^T leaves with each lane, for one row,
// the scores of tokens 4h .. 4h + 3 of every eight (h: the lane's half of the
// wave), and those are the tokens for which it then supplies the softmax
// weights as the right operand of out^T = V^T P^T; V's columns are read in
// the same order. A lane owns one row: the softmax needs no cross-lane work
// but one exchange between the two halves of a wave, and only when a score
// exceeds the running reference by 2^8.
//
// Bound by the matrix cores together with the vector instructions: a wave's
// tile of 32 rows and 64 tokens (head_dim 128) is 32 products of 32 cycles
// and 207 vector instructions, two waves share a SIMD, and under this load the
// clock is near 2.0 GHz. Of the time the matrix cores are busy 42 %, the vector
// units 39 % and LDS 31 %; one compute unit in seven waits for the last row
// tiles. Measured: a prompt of 4096 tokens, 32 query and 8 key-value heads of
// 128, bf16 cache: 142 to 156 us from card to card, 880 to 968 TFLOP/s of
// causal products (the library's product of 8192^3 reaches 1327); 8192 new
// tokens of 16384 with a window of 2048, MXFP4: 304 to 319 us. Tried and
// slower or equal: 64 rows a wave (199 and 392 us: copies to and from the
// accumulation registers), raised wave priority in either product, operands
// read 3 or 6 steps ahead, the barrier inside the second product, four of the
// eight waves half a turn behind the others (148 and 317 us).
#include "kv_device.h"
#include "kv_launch.h"

namespace qbn {
namespace {

using namespace kv;

constexpr int BN = 64;  // tokens per tile

struct PrefillArgs {
    Cache c;
    Batch b;
    const __bf16 *q;
    int64_t qt, qh;
    __bf16 *out;
    float *lse;
    int32_t *first;  // of more than kScanned sequences with cu [seqs + 1]: row tiles of those before; then, whether cu is out of order
    float *parts;  // [splits][tokens][heads][D] sums, then [splits][tokens][heads] references and weight sums
    float scale;   // |scale| times log2 e; q's sign bits are flipped where it is negative, and q is 0 where it is 0
    float far_unit;  // the power of two at or below `scale`
    uint32_t q_keep, q_flip;
    int group, window, sinks, splits, dim;
};

template <int F, int D, int NW>
struct Lay {
    static constexpr int NT = NW * 64, BM = NW * 32;
    // Bytes of a row in LDS (64 banks, 16 pieces of 16 bytes): an odd number of
    // pieces, so that sixteen rows' same piece lie in all banks, and 4 or 12
    // pieces (mod 16), so that four rows' 64 bytes do.
    static constexpr int KROW = 2 * D + 16, VROW = 2 * D + (D == 96 ? 0 : 64);
    static constexpr int KBUF = BN * KROW, VBUF = BN * VROW;  // one buffer each
    static constexpr int PER = D / 16;            // items (16 elements of a token's K and V) of a row
    static constexpr int ALL = BN * PER, ITEMS = (ALL + NT - 1) / NT;
    static constexpr int IB = 2 * kBits<F>, IW = IB / 4;  // bytes and words of an item
};

// The value, computed where this stands: the optimizer may not move it to its use.
template <typename T>
__device__ __forceinline__ T here(T v) {
    asm volatile("" : "+v"(v));
    return v;
}

// A sequence's new tokens, rows x to y of q; -1 where cu is out of order or leaves q.
__device__ __forceinline__ int new_tokens(const Batch &b, int x, int y) {
    return x >= 0 && y >= x && y <= b.tokens ? y - x : -1;
}

__device__ __forceinline__ int64_t row_tiles(int fresh, int group, int bm) {  // < 2^24
    return fresh < 0 ? 0 : ((int64_t)fresh * group + bm - 1) / bm;
}

// Many sequences: one workgroup lists the row tiles before each, and
// the others search the list.
constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void k_prefill_plan(PrefillArgs a, int bm) {
    __shared__ int64_t s_scan[kPlanThreads / 64 + 1];
    int64_t before = 0;
    bool wrong = false;
    for (int s0 = 0; s0 < a.b.seqs; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        int64_t all;
        const int n = s < a.b.seqs ? new_tokens(a.b, a.b.cu[s], a.b.cu[s + 1]) : 0;
        wrong |= n < 0;
        const int64_t at = block_scan<kPlanThreads>(row_tiles(n, a.group, bm), s_scan, all);
        if (s < a.b.seqs) a.first[s] = (int)min(before + at, (int64_t)0x7FFFFFFF);  // beyond the grid: cu is out of order
        before += all;
    }
    wrong = __syncthreads_or(wrong);
    if (threadIdx.x == 0) {
        a.first[a.b.seqs] = (int)min(before, (int64_t)0x7FFFFFFF);
        a.first[a.b.seqs + 1] = wrong;
    }
}

// The outputs of the rows of q that no sequence has, before cu[0] and from
// cu[seqs] on: 0 and -inf; of all rows NaN where cu is out of order. All
// workgroups of the grid share them.
template <int D>
__device__ __forceinline__ void write_rest(const PrefillArgs &a, int lo, int hi, bool wrong) {
    const int q_heads = a.c.heads * a.group;
    const int64_t total = (int64_t)a.b.tokens * q_heads, shift = total * blockIdx.y;
    const int64_t n = (int64_t)(wrong ? a.b.tokens : lo + (a.b.tokens - hi)) * q_heads;
    const float sum = wrong ? __builtin_nanf("") : 0.0f;
    float *st = a.parts + total * a.splits * D;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n * (D / 4); i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t k = i / (D / 4), row = wrong || k < (int64_t)lo * q_heads ? k : k + (int64_t)(hi - lo) * q_heads;
        const int d = (int)(i % (D / 4)) * 4;
        if (a.splits == 1) {
            *reinterpret_cast<u32x2 *>(a.out + row * D + d) = u32x2{pack2(sum, sum), pack2(sum, sum)};
            if (d == 0 && a.lse) a.lse[row] = wrong ? sum : kNegInf;
        } else {
            *reinterpret_cast<f32x4 *>(a.parts + (shift + row) * D + d) = f32x4{0, 0, 0, 0};
            if (d == 0) {
                st[shift + row] = kNegInf;
                st[total * a.splits + shift + row] = sum;
            }
        }
    }
}

// One element of V, as the tiles see it.
template <int F, int D>
__device__ __forceinline__ float element(const Cache &c, int64_t head, int ps, int slot, int d) {
    const int64_t at = (head * ps + slot) * D + d;
    uint32_t w[2] = {0, 0}, o[1];
    if constexpr (F == BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(c.v)[at] << 16);
    if constexpr (F == FP8) w[0] = c.v[at];
    if constexpr (F == FP4) w[0] = (c.v[at / 2] >> (4 * (d & 1))) & 15u;
    expand<F == BF16 ? FP8 : F, 2>(w, e8m0_operand(c.vs[(head * (D / 32) + d / 32) * ps + slot]), o);
    return __uint_as_float(o[0] << 16);
}

template <int F, int D, int NW>
__global__ __launch_bounds__(NW * 64, D <= 128 ? 2 : 1) void k_prefill(PrefillArgs a) {
    using L = Lay<F, D, NW>;
    __shared__ __align__(16) uint8_t s_k[2][L::KBUF], s_v[2][L::VBUF];
    __shared__ int s_odd;  // a tile that not every row sees held an infinity or NaN of V
    __shared__ int s_bad;  // a visible token's table entry was no page
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, half = lane >> 5;
    const int kv_head = blockIdx.x % a.c.heads;
    const int want = blockIdx.x / a.c.heads;  // row tile in the list of all sequences'

    // ---- which sequence and row tile (of a sequence's, the longest rows first)
    int b = a.b.seqs, tile = 0, q0 = 0, fresh = 0, len = 0;
    if (!a.b.cu) {  // one token each: as many tiles each
        const int each = (a.group + L::BM - 1) / L::BM;
        b = want / each, tile = each - 1 - want % each;
        if (b >= a.b.seqs) return;
        q0 = b, fresh = 1, len = length_of(a.b, b);
    } else {
        const int lo = start_of(a.b, 0), hi = start_of(a.b, a.b.seqs);
        bool wrong = false;
        if (a.first != nullptr) {
            wrong = a.first[a.b.seqs + 1] != 0;
            b = count_upto(a.first, a.b.seqs, want);
            if (b < a.b.seqs) {
                q0 = start_of(a.b, b);
                fresh = new_tokens(a.b, q0, start_of(a.b, b + 1));
                tile = (int)row_tiles(fresh, a.group, L::BM) - 1 - (want - a.first[b]);
                len = length_of(a.b, b);
            }
        } else {  // each wave scans the sequences for itself, 64 at a time, all loads in flight
            constexpr int CHUNKS = kScanned / 64;
            int x[CHUNKS], y[CHUNKS], l[CHUNKS], before = 0;
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                const int s = min(64 * i + lane, a.b.seqs - 1);
                if (i == 0 || 64 * i < a.b.seqs) x[i] = a.b.cu[s], y[i] = a.b.cu[s + 1], l[i] = a.b.lens[s];
            }
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                if (i > 0 && 64 * i >= a.b.seqs) break;
                const int n = 64 * i + lane < a.b.seqs ? new_tokens(a.b, x[i], y[i]) : 0;
                wrong |= __any(n < 0);
                const int upto = wave_scan((int)row_tiles(n, a.group, L::BM));
                const uint64_t here = __ballot(want >= before && want < before + upto);
                if (here) {
                    const int at = __builtin_ctzll(here);
                    b = 64 * i + at;
                    tile = before + __builtin_amdgcn_readlane(upto, at) - 1 - want;
                    q0 = __builtin_amdgcn_readlane(x[i], at);
                    fresh = __builtin_amdgcn_readlane(n, at);
                    len = __builtin_amdgcn_readlane(l[i], at);
                }
                before += __builtin_amdgcn_readlane(upto, 63);
            }
        }
        if (wrong || lo > 0 || hi < a.b.tokens) write_rest<D>(a, lo, hi, wrong);
        if (wrong || b >= a.b.seqs) return;
    }
    b = __builtin_amdgcn_readfirstlane(b), tile = __builtin_amdgcn_readfirstlane(tile);
    q0 = __builtin_amdgcn_readfirstlane(q0), fresh = __builtin_amdgcn_readfirstlane(fresh);
    len = __builtin_amdgcn_readfirstlane(len);
    const int rows = fresh * a.group;
    const int r0 = tile * L::BM;
    const int ps = 1 << a.c.page_shift;
    const bool bad = len < 0 || (((int64_t)len + ps - 1) >> a.c.page_shift) > a.b.row;
    if (bad) len = 0;
    // this lane's row; rows beyond the last repeat it and are not written
    const int r = r0 + wave * 32 + n;
    const bool mine = r < rows;
    const int rr = mine ? r : rows - 1, qi = rr / a.group, head = kv_head * a.group + rr % a.group;
    const int pos = len - fresh + qi;
    const int pmin = len - fresh + r0 / a.group;
    const int pmax = len - fresh + (min(r0 + L::BM, rows) - 1) / a.group;
    // keys that some row of the workgroup sees: the sinks, then from lo to pmax
    const int lo = a.window > 0 && pmin >= a.window ? pmin - a.window + 1 : 0;
    const int first = lo / BN, sink_tiles = min((min(a.sinks, lo) + BN - 1) / BN, first);
    const int all = bad || pmax < 0 ? 0 : sink_tiles + pmax / BN + 1 - first;
    const int u0 = (int)((int64_t)all * blockIdx.y / a.splits), u1 = (int)((int64_t)all * (blockIdx.y + 1) / a.splits);

    bf16x8 q[D / 16];
    {
        const __bf16 *row = a.q + (int64_t)(q0 + qi) * a.qt + (int64_t)head * a.qh + 8 * half;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            u32x4 t = ld16(row + 16 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = (t[i] & a.q_keep) ^ a.q_flip;
            q[k] = as_bf16x8(t);
        }
    }
    f32x16 acc[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t) acc[t] = f32x16{};
    Reference running = {kNegInf, a.scale};
    float sum = 0.0f;

    // Conditions without short circuits: as branches they cost more than they save.
    const auto tile_token = [&](int u) { return (u < sink_tiles ? u : u - sink_tiles + first) * BN; };
    const auto token_after = [&](int t0) { return t0 + BN == sink_tiles * BN ? first * BN : t0 + BN; };
    // tokens that every row of the workgroup sees need no mask
    const auto is_edge = [&](int t0) {
        return (int)(t0 + BN - 1 > pmin) | ((int)(a.window > 0) & (int)(t0 <= pmax - a.window) & (int)(t0 + BN > a.sinks));
    };
    const auto is_seen = [&](int t) { return (t <= pmax) & ((t >= lo) | (t < a.sinks)); };

    // ---- a thread's part of a tile: its items' page table entries, bytes and scales
    const int32_t *row_table = a.b.table + (int64_t)b * a.b.row_stride;
    const auto item = [&](int i, int &t, int &blk) {
        int it = tid + i * L::NT;
        if (L::ALL % L::NT) it = min(it, L::ALL - 1);  // threads without an item repeat the last
        t = it / L::PER, blk = it % L::PER;
    };
    struct Items {
        uint32_t w[L::ITEMS][L::IW], sc[L::ITEMS];
    };
    struct Entries {
        uint32_t page[L::ITEMS];
    };
    Items rk, rv;
    constexpr int ROW = D * kBits<F> / 8;  // bytes
    const uint32_t page_rows = (uint32_t)a.c.heads << a.c.page_shift;
    const int64_t head_rows = (int64_t)kv_head << a.c.page_shift;
    const uint8_t *k_head = a.c.k + head_rows * ROW, *v_head = a.c.v + head_rows * ROW;
    const uint8_t *ks_head = a.c.ks + head_rows * (D / 32), *vs_head = a.c.vs + head_rows * (D / 32);
    // Unconditional loads, here and below: behind a branch the compiler could
    // not tell which are in flight, and would wait for all of them. Tokens
    // beyond the last visible one stand for that one.
    const auto look_up = [&](int i, int t0, Entries &e) {
        int t, blk;
        item(i, t, blk);
        const uint32_t at = (uint32_t)min(t0 + t, pmax) >> a.c.page_shift;
        e.page[i] = *reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(row_table) + at * 4);
    };
    const auto load = [&](int i, const uint8_t *elements, const uint8_t *scales, int t0, const Entries &from, Items &r) {
        int t, blk;
        item(i, t, blk);
        uint32_t page = from.page[i];
        if (__any(page >= (uint32_t)a.c.pages)) {
            if (page >= (uint32_t)a.c.pages) {
                if (is_seen(t0 + t)) s_bad = 1;
                page = 0;
            }
        }
        const uint32_t slot = (uint32_t)(t0 + t) & (uint32_t)(ps - 1);
        load_words<L::IB>(elements + blk * L::IB + slot * ROW + (uint64_t)page * (page_rows * ROW), r.w[i]);
        if constexpr (F != BF16)
            r.sc[i] = scales[((blk / 2) << a.c.page_shift) + slot + (uint64_t)page * (page_rows * (D / 32))];
    };
    const auto expand_item = [&](const Items &r, int i, uint32_t (&x)[2][4]) {
        const float f = F == BF16 ? 1.0f : e8m0_operand(r.sc[i]);
#pragma unroll
        for (int e = 0; e < 2; ++e) expand8<F>(r.w[i] + e * (L::IW / 2), f, x[e]);
    };
    const auto put = [&](uint8_t *d, const uint32_t (&x)[2][4]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) *reinterpret_cast<u32x4 *>(d + 16 * e) = u32x4{x[e][0], x[e][1], x[e][2], x[e][3]};
    };
    const auto store_k = [&](const Items &r, int i, int buf) {
        int t, blk;
        item(i, t, blk);
        uint32_t x[2][4];
        expand_item(r, i, x);
        put(s_k[buf] + t * L::KROW + blk * 32, x);
    };
    const auto store_v = [&](int i, int t0, bool edge, int buf) {
        int t, blk;
        item(i, t, blk);
        uint32_t x[2][4];
        expand_item(rv, i, x);
        if (edge) {  // what no row sees becomes 0; what only some see is looked over
            const bool on = is_seen(t0 + t);
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[e][j] = on ? x[e][j] : 0u;
                    odd |= (x[e][j] & 0x7F80u) == 0x7F80u || (x[e][j] & 0x7F800000u) == 0x7F800000u;
                }
            if (__any(odd)) {  // taken out of the product; put where they belong at the end
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[e][j] &= (x[e][j] & 0x7F80u) == 0x7F80u ? 0xFFFF0000u : 0xFFFFFFFFu;
                        x[e][j] &= (x[e][j] & 0x7F800000u) == 0x7F800000u ? 0x0000FFFFu : 0xFFFFFFFFu;
                    }
                s_odd = 1;
            }
        }
        put(s_v[buf] + t * L::VROW + blk * 32, x);
    };

    struct Scores {
        f32x16 s[2];
    };
    const int koff = n * L::KROW + 16 * half;
    const int voff = (4 * half + (lane & 15) / 4) * L::VROW + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    // Matrix operands, read from LDS in the order of the products' steps.
    constexpr int SK = D / 8, SV = D / 8, AHEAD = 4;
    const auto k_part = [&](int buf, int i) { return as_bf16x8(ld16(s_k[buf] + koff + i % 2 * 32 * L::KROW + 32 * (i / 2))); };
    const auto v_part = [&](int buf, int i) {
        const uint8_t *v = s_v[buf] + voff + 16 * (i / (D / 32)) * L::VROW + 64 * (i % (D / 32));
        const u32x2 lo = ld_tr16(v), hi = ld_tr16(v + 8 * L::VROW);
        return as_bf16x8(u32x4{lo.x, lo.y, hi.x, hi.y});
    };
    const auto k_step = [&](Scores &x, int i, bf16x8 part) {
        if (i < 2) x.s[i] = f32x16{};
        x.s[i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(part, q[i / 2], x.s[i % 2], 0, 0, 0);
    };
    struct Weights {
        u32x4 p[4];
    };
    const auto v_step = [&](const Weights &w, int i, bf16x8 part) {
        const int t = i % (D / 32), g = i / (D / 32);
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(part, as_bf16x8(w.p[g]), acc[t], 0, 0, 0);
    };
    // Word k of the weights is made of scores 2k and 2k + 1, in three ticks, so
    // that nothing waits for the exponential before it: tick k scales the
    // scores, tick k + 1 takes the powers, tick k + 2 adds and rounds: to
    // bfloat16 for the product with V (2^-8 of a weight at most; an output is off
    // from binary64 by 1.1 to 1.4 times as much as with binary32 weights, which
    // would need two products in place of one), while the sum takes them as they are.
    float arg[2][2], pow[2][2];
    const auto tick = [&](const Scores &x, float base, Weights &w, int k) {
        if (k >= 1 && k <= 16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) pow[(k - 1) % 2][i] = here(exp2_fast(arg[(k - 1) % 2][i]));
        }
        if (k >= 2) {
            const float y = pow[k % 2][0], z = pow[k % 2][1];
            sum = here(sum + (y + z));
            w.p[(k - 2) / 4][(k - 2) % 4] = here(pack2(y, z));
        }
        if (k < 16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) arg[k % 2][i] = here(__builtin_fmaf(x.s[k / 8][2 * k % 16 + i], running.unit, -base));
        }
    };
    const auto larger = [&](const Scores &x, float top, int i) {
        return here(__builtin_fmaxf(top, __builtin_fmaxf(x.s[i / 8][2 * i % 16], x.s[i / 8][2 * i % 16 + 1])));
    };
    // Masks the scores of an edge and raises the reference where they exceed it.
    const auto settle = [&](Scores &x, float top, int t0, bool edge) {
        if (edge) {
            top = kNegInf;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int k = t0 + 32 * t + 8 * (e / 4) + 4 * half + e % 4;
                    const bool on = (k <= pos) & ((a.window == 0) | (k > pos - a.window) | (k < a.sinks));
                    x.s[t][e] = on ? x.s[t][e] : kNegInf;
                    top = __builtin_fmaxf(top, x.s[t][e]);
                }
        }
        if (__any(top * running.unit > running.at + 8.0f)) {
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            const float f = raise(running, top, a.scale, a.far_unit);
            sum *= f;
#pragma unroll
            for (int t = 0; t < D / 32; ++t) acc[t] *= f;
        }
    };
    if (tid == 0) s_odd = s_bad = 0;
    __syncthreads();
    // K runs a tile ahead of V in LDS: the scores of the next tile are computed
    // next to the exponentials of this one.
    if (u0 < u1) {
        const int t0 = tile_token(u0);
        int t1 = token_after(t0), t2 = token_after(t1);  // the next two tiles
        Entries e0, e1;
        const auto look_up_all = [&](int t, Entries &e) {
#pragma unroll
            for (int i = 0; i < L::ITEMS; ++i) look_up(i, t, e);
        };
        const auto load_all = [&](const uint8_t *elements, const uint8_t *scales, int t, const Entries &e, Items &r) {
#pragma unroll
            for (int i = 0; i < L::ITEMS; ++i) load(i, elements, scales, t, e, r);
        };
        look_up_all(t0, e0);
        look_up_all(t1, e1);
        Items k0;
        load_all(k_head, ks_head, t0, e0, k0);
        load_all(v_head, vs_head, t0, e0, rv);
        load_all(k_head, ks_head, t1, e1, rk);
#pragma unroll
        for (int i = 0; i < L::ITEMS; ++i) {
            store_k(k0, i, 0);
            store_v(i, t0, is_edge(t0), 0);
            store_k(rk, i, 1);
        }
        look_up_all(t2, e0);
        load_all(v_head, vs_head, t1, e1, rv);
        __syncthreads();
        Scores s0, s1;
        float top = kNegInf;
#pragma unroll
        for (int i = 0; i < SK; ++i) k_step(s0, i, k_part(0, i));
#pragma unroll
        for (int i = 0; i < 16; ++i) top = larger(s0, top, i);
        settle(s0, top, t0, is_edge(t0));
        __syncthreads();  // the first turn overwrites the first K
        // One tile: its scores are in x, the next one's go to y; e holds the page
        // entries of tile t2, f gets those of the one after it. The vector work
        // is spread evenly over the products' steps, whose order the scheduling
        // barriers keep: two waves share a SIMD, and where both are in a part
        // with much of it the matrix core waits. Next to the products with K
        // stand the first EARLY ticks of the weights and K's loads, next to
        // V's the other ticks, then the maximum, the stores to LDS and V's
        // loads. Operands are read AHEAD steps before their use.
        constexpr int TICKS = 18, EARLY = 11, HALF = SV / 2;
        const auto turn = [&](int buf, Scores &x, Scores &y, Entries &e, Entries &f) {
            const int t3 = token_after(t2);
            const bool edge = is_edge(t1);
            // One wave on a SIMD: the half of its 512 registers that only matrix
            // instructions and copies reach holds what only matrix instructions
            // use. Left to itself the compiler puts the scores there and stores
            // others to memory (4096 tokens, 32 / 8 heads, bf16: 256 wide 599 us,
            // so 349; 192 wide 285, so 272).
            if constexpr (D > 128) {
#pragma unroll
                for (int t = 0; t < D / 32; ++t) asm volatile("" : "+a"(acc[t]));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) asm volatile("" : "+a"(q[k]));
            }
            const float base = running.at == kNegInf ? 0.0f : running.at;
            Weights w;
            bf16x8 part[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) part[i] = k_part(buf ^ 1, i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < SK; ++i) {
                k_step(y, i, part[i % AHEAD]);
                part[i % AHEAD] = i + AHEAD < SK ? k_part(buf ^ 1, i + AHEAD) : v_part(buf, i + AHEAD - SK);
                if (i < L::ITEMS) look_up(i, t3, f);
                else if (i < 2 * L::ITEMS) load(i - L::ITEMS, k_head, ks_head, t2, e, rk);
#pragma unroll
                for (int k = EARLY * i / SK; k < EARLY * (i + 1) / SK; ++k) tick(x, base, w, k);
                __builtin_amdgcn_sched_barrier(0);
            }
            float top = kNegInf;
#pragma unroll
            for (int i = 0; i < SV; ++i) {
                v_step(w, i, part[i % AHEAD]);
                if (i + AHEAD < SV) part[i % AHEAD] = v_part(buf, i + AHEAD);
                if (i < HALF) {
#pragma unroll
                    for (int k = EARLY + (TICKS - EARLY) * i / HALF; k < EARLY + (TICKS - EARLY) * (i + 1) / HALF; ++k)
                        tick(x, base, w, k);
                } else {
#pragma unroll
                    for (int k = 16 * (i - HALF) / HALF; k < 16 * (i + 1 - HALF) / HALF; ++k) top = larger(y, top, k);
                    const int j = i - HALF;  // HALF is 4 * ITEMS, or 3 * ITEMS at 96
                    if (j < L::ITEMS) store_v(j, t1, edge, buf ^ 1);
                    else if (j < 2 * L::ITEMS) load(j - L::ITEMS, v_head, vs_head, t2, e, rv);
                    else if (j < 3 * L::ITEMS) store_k(rk, j - 2 * L::ITEMS, buf);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            settle(y, top, t1, edge);
            t1 = t2, t2 = t3;
            __syncthreads();
        };
        const auto last = [&](int buf, Scores &x) {
            const float base = running.at == kNegInf ? 0.0f : running.at;
            Weights w;
#pragma unroll
            for (int k = 0; k < TICKS; ++k) tick(x, base, w, k);
#pragma unroll
            for (int i = 0; i < SV; ++i) v_step(w, i, v_part(buf, i));
        };
        int u = u0;
        for (; u + 2 < u1; u += 2) {
            turn(0, s0, s1, e0, e1);
            turn(1, s1, s0, e1, e0);
        }
        if (u + 1 < u1) {
            turn(0, s0, s1, e0, e1);
            last(1, s1);
        } else {
            last(0, s0);
        }
    }

    const float ref = scaled(running, a.scale);
    sum += __shfl_xor(sum, 32);
    if (bad || s_bad) sum = __builtin_nanf("");
    const int64_t total = (int64_t)a.b.tokens * (a.c.heads * a.group), shift = total * blockIdx.y;
    const int64_t row = (int64_t)(q0 + qi) * (a.c.heads * a.group) + head;
    if (mine && a.splits == 1) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<u32x2 *>(a.out + row * D + 32 * t + 8 * i + 4 * half) =
                    u32x2{pack2(acc[t][4 * i] * inv, acc[t][4 * i + 1] * inv),
                          pack2(acc[t][4 * i + 2] * inv, acc[t][4 * i + 3] * inv)};
        if (half == 0 && a.lse) a.lse[row] = sum == 0.0f ? kNegInf : (ref + __builtin_amdgcn_logf(sum)) * kLn2;
    } else if (mine) {
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f32x4 *>(a.parts + (shift + row) * D + 32 * t + 8 * i + 4 * half) =
                    f32x4{acc[t][4 * i], acc[t][4 * i + 1], acc[t][4 * i + 2], acc[t][4 * i + 3]};
        if (half == 0) {
            float *st = a.parts + total * a.splits * D;
            st[shift + row] = ref;
            st[total * a.splits + shift + row] = sum;
        }
    }
    // Infinities and NaN of V in tiles that not every row sees: added to the
    // rows that see them, after the sums are written. A thread owns an element
    // of the head, so that no two add to the same output.
    if (s_odd == 0) return;
    __syncthreads();
    for (int u = u0; u < u1; ++u) {
        const int t0 = tile_token(u);
        if (!is_edge(t0) || tid >= D) continue;
        for (int t = t0; t < t0 + BN; ++t) {
            if (!is_seen(t)) continue;
            const int p = a.b.table[(int64_t)b * a.b.row_stride + (t >> a.c.page_shift)];
            if ((uint32_t)p >= (uint32_t)a.c.pages) continue;
            const int64_t h = (int64_t)p * a.c.heads + kv_head;
            const int slot = t & (ps - 1);
            const float v = element<F, D>(a.c, h, ps, slot, tid);
            if (__builtin_isfinite(v)) continue;
            const float add = __builtin_isnan(v) ? v : __builtin_copysignf(__builtin_huge_valf(), v);
            for (int k = r0; k < min(r0 + L::BM, rows); ++k) {
                const int pk = len - fresh + k / a.group;
                if (t > pk || (a.window > 0 && t <= pk - a.window && t >= a.sinks)) continue;
                const int64_t o = ((int64_t)(q0 + k / a.group) * (a.c.heads * a.group) + kv_head * a.group + k % a.group);
                if (a.splits == 1) a.out[o * D + tid] = (__bf16)((float)a.out[o * D + tid] + add);
                else a.parts[(shift + o) * D + tid] += add;
            }
        }
    }
}

// Joins the pieces of a split length, in order: D / 4 lanes per row, eight
// pieces in flight. Bound by the pieces' bytes.
template <int D>
__global__ __launch_bounds__(256) void k_prefill_join(PrefillArgs a, int64_t total) {
    constexpr int L = D / 4, ROWS = 64 / L;  // lanes of a row, rows of a wave
    const int lane = threadIdx.x & 63, d = lane % L * 4;
    const int64_t row = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * ROWS + lane / L;
    if (lane >= ROWS * L || row >= total) return;
    const float *st = a.parts + total * a.splits * D;
    float top = kNegInf, sum = 0.0f;
    f32x4 o = {0, 0, 0, 0};
    for (int i0 = 0; i0 < a.splits; i0 += 8) {
        f32x4 v[8];
        float r[8], s[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t at = min(i0 + k, a.splits - 1) * total + row;
            v[k] = *reinterpret_cast<const f32x4 *>(a.parts + at * D + d);
            r[k] = st[at];
            s[k] = st[a.splits * total + at];
        }
        float now = top;
#pragma unroll
        for (int k = 0; k < 8; ++k) now = __builtin_fmaxf(now, r[k]);
        const float f = top == now ? 1.0f : exp2_fast(top - now);
        o *= f;
        sum *= f;
        top = now;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i0 + k < a.splits) {
                const float w = r[k] == top ? 1.0f : exp2_fast(r[k] - top);
                o += v[k] * w;
                sum += s[k] * w;
            }
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    *reinterpret_cast<u32x2 *>(a.out + row * D + d) = u32x2{pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv)};
    if (d == 0 && a.lse) a.lse[row] = sum == 0.0f ? kNegInf : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

struct Plan {
    int64_t tiles;  // row tiles at most
    int splits, waves;
};

Plan plan_of(const qbn_kv_cache &c, const qbn_kv_batch &b, int q_heads, int window, int sinks) {
    Plan p;
    const int64_t group = q_heads / c.heads;
    // Tiles of 256 rows where they fill the compute units and a sequence has more
    // than 128 on the average. Tiles of 256 and of 128, us: MXFP8, 32 / 8 heads of
    // 128 on 2048 tokens, 160 sequences of 64 rows 344 and 216, 80 of 128 202 and
    // 133, 64 of 160 142 and 156, 51 of 200 133 and 143, 42 of 240 130 and 119 (of
    // 64 93 and 74); 65536 of one row, 4 heads of 64, 6.6 ms and 3.1.
    p.waves = c.head_dim <= 128 && b.tokens * group / 256 * c.heads >= 256 && b.tokens * group > 128 * b.seqs ? 8 : 4;
    const int BM = p.waves * 32;
    p.tiles = b.cu ? b.tokens * group / BM + b.seqs : b.seqs * ((group + BM - 1) / BM);
    int64_t units = (b.row * c.page_size + BN - 1) / BN;
    if (window > 0) {
        const int64_t seen = ((int64_t)window + BM / group) / BN + 2 + ((int64_t)sinks + BN - 1) / BN;
        if (seen < units) units = seen;
    }
    const int64_t blocks = p.tiles * c.heads;
    // Few row tiles: the length is split until about one workgroup per compute
    // unit runs, each with at least two tiles of 64 tokens. For about 128, 256,
    // 512 and 1024 workgroups, us with the join: chunks of up to 341 tokens on
    // 1531, 12 / 4 heads of 96 MXFP8 36, 25, 27, 32; 4 of 64 on 2048, 32 / 8 of
    // 128 bf16 46, 33, 31, 38; 128 and 16 on 8192 and 200, 8 / 1 of 64 MXFP4
    // 22, 20, 24, 31; 3 of 500 on 1000, 8 / 4 of 256 50, 43, 55, 82; 8 of 32 on
    // 4096, 16 / 2 of 128 50, 29, 32, 40; but 256 on 30000, 32 / 8 of 128 MXFP8
    // 618, 219, 155, 167, and 16 of 16 on 4096, MXFP4 94, 94, 74, 58.
    int64_t splits = blocks > 0 && blocks < 256 ? 256 / blocks : 1;
    if (splits > units / 2) splits = units / 2;
    p.splits = (int)(splits < 1 ? 1 : splits > 64 ? 64 : splits);
    return p;
}

int64_t part_bytes(const Plan &p, const qbn_kv_cache &c, const qbn_kv_batch &b, int q_heads) {
    return p.splits > 1 ? p.splits * b.tokens * q_heads * ((int64_t)c.head_dim + 2) * 4 : 0;
}
bool listed(const qbn_kv_batch &b) { return b.cu && b.seqs > kScanned; }

template <int F>
hipError_t launch(const PrefillArgs &a, dim3 grid, int waves, hipStream_t s) {
    const int64_t total = (int64_t)a.b.tokens * a.c.heads * a.group;
#define QBN_KV_DIM(DD)                                                         \
    case DD:                                                                   \
        if (DD <= 128 && waves == 8) k_prefill<F, DD, DD <= 128 ? 8 : 4><<<grid, 512, 0, s>>>(a); \
        else k_prefill<F, DD, 4><<<grid, 256, 0, s>>>(a);                      \
        if (a.splits > 1) {                                                    \
            constexpr int per = 4 * (256 / DD);                                \
            k_prefill_join<DD><<<(unsigned)((total + per - 1) / per), 256, 0, s>>>(a, total); \
        }                                                                      \
        break;
    if (a.first) k_prefill_plan<<<1, kPlanThreads, 0, s>>>(a, waves * 32);
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

int64_t kv_prefill_workspace(const qbn_kv_cache &c, const qbn_kv_batch &b, int q_heads, int window, int sinks) {
    const Plan p = plan_of(c, b, q_heads, window, sinks);
    if (p.tiles * c.heads >= kGridThreads / (p.waves * 64)) return -1;
    return part_bytes(p, c, b, q_heads) + (listed(b) ? 4 * (b.seqs + 2) : 0);
}

hipError_t launch_kv_prefill(const qbn_kv_cache &c, int64_t layer, const qbn_kv_batch &b, int q_heads, const KvRows &q,
                             float scale, int window, int sinks, void *out, float *lse, void *ws, hipStream_t s) {
    const Plan p = plan_of(c, b, q_heads, window, sinks);
    const int64_t elems = layer * c.pages * c.heads * c.page_size * c.head_dim;
    const int bits = c.format == QBN_KV_BF16 ? 16 : c.format == QBN_MXFP8 ? 8 : 4;
    PrefillArgs a;
    a.c = {(const uint8_t *)c.k + elems * bits / 8, (const uint8_t *)c.v + elems * bits / 8,
           (const uint8_t *)c.k_scales + elems / 32, (const uint8_t *)c.v_scales + elems / 32, c.heads,
           __builtin_ctz(c.page_size), (int)c.pages};
    a.b = {(int)b.seqs, (int)b.tokens, (int)b.row, b.row_stride, b.table, b.lens, b.cu};
    a.q = (const __bf16 *)q.p;
    a.qt = q.token_stride, a.qh = q.head_stride;
    a.out = (__bf16 *)out, a.lse = lse;
    a.parts = (float *)ws;
    a.first = listed(b) ? (int32_t *)((uint8_t *)ws + part_bytes(p, c, b, q_heads)) : nullptr;
    a.scale = scale == 0.0f ? 1.0f : fabsf(scale) * kLog2e;
    a.far_unit = ldexpf(1.0f, ilogbf(a.scale));
    a.q_keep = scale == 0.0f ? 0u : ~0u;
    a.q_flip = scale < 0.0f ? 0x80008000u : 0u;
    a.group = q_heads / c.heads, a.window = window, a.sinks = sinks, a.splits = p.splits, a.dim = c.head_dim;
    const dim3 grid((unsigned)(p.tiles * c.heads), (unsigned)p.splits);
    if (c.format == QBN_KV_BF16) return launch<BF16>(a, grid, p.waves, s);
    return c.format == QBN_MXFP8 ? launch<FP8>(a, grid, p.waves, s) : launch<FP4>(a, grid, p.waves, s);
}

}  // namespace qbn
