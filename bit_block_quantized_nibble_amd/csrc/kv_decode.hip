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
// Splitting. A workgroup takes a piece of one (sequence, head group) pair. How
// many units of 128 tokens a piece has follows from the lengths: so many that
// about `blocks` pieces come out of all pairs, whatever the lengths. The
// pieces of a pair are alike; each workgroup finds its own by a scan of the
// lengths, of many sequences by a search of the list that a first
// kernel makes of them. A pair of one piece is written at once; the pieces of the others go
// through the workspace, where the first of them notes which they are, and a
// second kernel joins them in order. (Pieces that
// run over the end of a pair into the next one would be more even, but the
// workgroups that hold an end then pass twice through the chain of length,
// page table, first tile and output, and that chain is most of a short call.)
//
// Measured (kernel and join, one layer): 32 sequences of up to 4096 tokens, 8
// heads of 128, MXFP8 (100 MB): 23.1 + 4.2 us, 4.3 TB/s in the first; two of
// up to 131072 tokens, MXFP4 (179 MB): 36.8 + 4.7 us, 4.9 TB/s, what a copy of
// 2 GiB reaches (4.95); 64 with a window of 4096 and one head of 64, MXFP4
// (15 MB): 10.6 + 4.1 us, of which 4 are the chain of launch, lengths, table,
// first tile and output, and the rest is instruction issue. Tried and slower: three or four
// tiles in flight (batch 28.9 -> 32.6 us), 1024 pieces instead of 512 (long
// 37.4 -> 39.7), and the join inside this kernel by the workgroup that
// finishes last (long 41.4 -> 46.4, though window 12.8 -> 11.8).
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
    float *parts;  // pieces: [16][D] sums, then [16] maxima and [16] sums of weights
    int2 *found;   // per pair: its first piece, how many there are
    int32_t *first;  // of more than kScanned sequences [seqs + 1]: pieces (of a pair) of those before
    float scale;   // |scale| times log2 e; q's sign bits are flipped where it is negative, and q is 0 where it is 0
    float far_unit;  // the power of two at or below `scale`
    uint32_t q_keep, q_flip;
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

// Pieces of a pair of n units; a sequence without tokens has outputs to be written, too.
__device__ __forceinline__ uint32_t pieces_of(int n, uint32_t per) { return n == 0 ? 1 : ((uint32_t)n + per - 1) / per; }

// Units of a piece at most, from the units of all sequences: about `blocks`
// pieces of all pairs. Rounded up pair by pair, that may be a few pieces more
// than run at once, and those would double the time: longer pieces, until
// all fit. count(per): the pieces of all sequences (fewer than 2^31 / rows).
template <typename Count>
__device__ __forceinline__ uint32_t plan_pieces(const DecodeArgs &a, int64_t total, Count count) {
    const int64_t most = div_i64(total * a.rows + a.blocks - 1, a.blocks);
    uint32_t per = (uint32_t)(most < 1 ? 1 : most < (1 << 24) ? most : 1 << 24);
    for (int i = 0; i < 8 && (int64_t)a.b.seqs * a.rows <= a.blocks; ++i) {
        const int64_t pieces = count(per) * a.rows;
        if (pieces <= a.blocks) break;
        per = max(per + 1, (uint32_t)div_i64(per * pieces + a.blocks - 1, a.blocks));
    }
    return per;
}

// Units and pieces of the sequences, 64 at a time: each wave scans the lengths
// for itself, which costs a load and a few lane moves and no barrier.
struct Chunk {
    int len, n, upto, all;  // of this lane's sequence: its length, its pieces; pieces up to and with it, of all 64
};
__device__ __forceinline__ int length_at(const DecodeArgs &a, int s0) {  // of this lane's sequence
    const int s = s0 + (threadIdx.x & 63);
    return s < a.b.seqs ? a.b.lens[s] : 0;
}
__device__ __forceinline__ Chunk pieces_at(const DecodeArgs &a, int s0, int len, uint32_t per) {
    Chunk c;
    c.len = len;
    c.n = s0 + (int)(threadIdx.x & 63) < a.b.seqs ? (int)pieces_of(span_of(a, len).n, per) : 0;
    c.upto = wave_scan(c.n);
    c.all = __builtin_amdgcn_readlane(c.upto, 63);
    return c;
}

struct Plan {
    Chunk first;   // of sequences 0 .. 63
    uint32_t per;  // units of a piece at most
};
__device__ __forceinline__ Plan plan_units(const DecodeArgs &a) {
    Plan p;
    const int len = length_at(a, 0);
    const auto units = [&](int len) { return __builtin_amdgcn_readlane(wave_scan(span_of(a, len).n), 63); };  // each less than 2^24
    int64_t total = units(len);
    for (int s = 64; s < a.b.seqs; s += 64) total += units(length_at(a, s));
    const auto count = [&](uint32_t per) {
        p.first = pieces_at(a, 0, len, per);
        int64_t n = p.first.all;
        for (int s = 64; s < a.b.seqs; s += 64) n += pieces_at(a, s, length_at(a, s), per).all;
        return n;
    };
    p.per = plan_pieces(a, total, count);
    p.first = pieces_at(a, 0, len, p.per);
    return p;
}

// Many sequences: one workgroup lists the pieces before each sequence, and the
// others search the list.
constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void k_decode_plan(DecodeArgs a) {
    __shared__ int64_t s_scan[kPlanThreads / 64 + 1];
    const auto sum = [&](int64_t mine) {
        int64_t total;
        block_scan<kPlanThreads>(mine, s_scan, total);
        return total;
    };
    int64_t mine = 0;
    for (int s = threadIdx.x; s < a.b.seqs; s += kPlanThreads) mine += span_of(a, a.b.lens[s]).n;
    const uint32_t per = plan_pieces(a, sum(mine), [&](uint32_t per) {
        int64_t n = 0;
        for (int s = threadIdx.x; s < a.b.seqs; s += kPlanThreads) n += pieces_of(span_of(a, a.b.lens[s]).n, per);
        return sum(n);
    });
    int64_t before = 0;
    for (int s0 = 0; s0 < a.b.seqs; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        int64_t all;
        const int64_t at = block_scan<kPlanThreads>(s < a.b.seqs ? pieces_of(span_of(a, a.b.lens[s]).n, per) : 0, s_scan, all);
        if (s < a.b.seqs) a.first[s] = (int)(before + at);  // fewer than the main kernel's workgroups
        before += all;
    }
    if (threadIdx.x == 0) a.first[a.b.seqs] = (int)before;
}

// A wave's 32 tokens as loaded. A vector memory instruction takes a compute
// unit's address unit 16 cycles whatever its width, so loads are 16 bytes a lane
// where they can be: V and the scales go through LDS (the wave's own part, no
// barrier), where the narrow pieces that the matrix operands are made of cost
// a quarter. K's pieces are 16 bytes, but 8 (MXFP4 at 64 and 192, MXFP8 at 96)
// or 4 (MXFP4 at 96) where the row has no more for a lane group: 32 sequences
// of 4096 tokens, MXFP4, 3.1 TB/s at 64 and 96 against 4.3 at 128.
template <int F, int D>
struct Tile {
    static constexpr int ROW = D * kBits<F> / 8;  // bytes of a token's head
    // K: a lane group's contiguous piece of E elements, NC pieces per row
    static constexpr int E = F == FP4 ? (D % 128 == 0 ? 32 : D % 64 == 0 ? 16 : 8) : F == FP8 ? (D % 64 == 0 ? 16 : 8) : 8;
    static constexpr int NC = D / (4 * E);
    static constexpr int KB = E * kBits<F> / 8, KW = KB / 4;
    // V: 16 lanes cover 128, 64 or 32 elements of a row
    static constexpr int N8 = D / 128, N4 = D % 128 / 64, N2 = D % 64 / 32, NS = N8 + N4 + N2;
    static constexpr int words(int w) { return w * kBits<F> / 32 > 0 ? w * kBits<F> / 32 : 1; }
    static constexpr int W8 = words(8), W4 = words(4), W2 = words(2), VW = N8 * W8 + N4 * W4 + N2 * W2;
    static constexpr bool STAGED = F != BF16 || D % 128 != 0;  // otherwise V's pieces are 16 bytes already
    static constexpr int CHUNKS = 2 * ROW, VN = (CHUNKS + 63) / 64;           // 16-byte chunks of 32 rows; loads
    static constexpr int SCALES = F == BF16 ? 0 : D / 2, SN = (SCALES + 63) / 64;  // 4-byte words of K's and V's scales; loads
    // In LDS: V's rows with 16 bytes of padding, then the scales [K, V][D / 32][32].
    static constexpr int VROW = ROW + 16, SOFF = STAGED ? 32 * VROW : 0, BYTES = SOFF + 4 * SCALES;
    uint32_t k[2][NC * KW];
    u32x4 v[STAGED ? VN : 8 * N8];
    uint32_t s[SN > 0 ? SN : 1];
};

template <int F, int D>
struct Decoder {
    using T = Tile<F, D>;
    static constexpr int ROW = T::ROW;
    const DecodeArgs &a;
    uint8_t *const lds;  // the wave's part
    int m, g, b, lane;
    Span sp;
    // this head in page 0: K's first bytes of this lane, V's and the scales' first
    const uint8_t *k, *v, *ks, *vs;
    uint32_t page_rows;
    bool bad = false;

    __device__ __forceinline__ Decoder(const DecodeArgs &args, uint8_t *part, int lane, int seq, int kv_head, int len)
        : a(args), lds(part), m(lane & 15), g(lane >> 4), b(seq), lane(lane), sp(span_of(args, len)) {
        const int ps = 1 << a.c.page_shift;
        page_rows = (uint32_t)a.c.heads << a.c.page_shift;  // a page's bytes fit 32 bits
        const int64_t head = (int64_t)kv_head << a.c.page_shift;
        // K: rows 4g' + i of the first product are tokens 8g' + i, of the second 8g' + 4 + i
        const int kt = (8 * (m / 4) + m % 4) & (ps - 1);
        k = a.c.k + (head + kt) * ROW + g * T::KB;
        v = a.c.v + head * ROW;
        ks = a.c.ks + head * (D / 32);
        vs = a.c.vs + head * (D / 32);
    }

    __device__ __forceinline__ bool sees(int t) const { return (t < sp.len) & ((t >= sp.lo) | (t < a.sinks)); }

    // The pages of tokens t .. t + 15 and t + 16 .. t + 31 (t % 32 == 0): page 0
    // where none of them is seen.
    struct Pages {
        uint32_t p[2];
    };
    __device__ __forceinline__ Pages pages_of(int t0) {
        Pages r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + 16 * i;
            const bool any = (t < sp.len) & ((t + 15 >= sp.lo) | (t < a.sinks));
            const uint32_t p = table_entry(a.b, b, any ? t >> a.c.page_shift : 0);
            const bool page = p < (uint32_t)a.c.pages;
            bad |= any & !page;
            r.p[i] = (any & page) ? p : 0;
        }
        return r;
    }

    __device__ __forceinline__ void load(T &r, int t0, Pages pages) {
        const int ps = 1 << a.c.page_shift;
        const uint32_t slot = (uint32_t)t0 & (uint32_t)(ps - 1);  // 0 where a page holds half a tile
        {
            const uint32_t page = m < 8 ? pages.p[0] : pages.p[1];
            const uint8_t *row = k + (uint64_t)page * (page_rows * ROW) + slot * ROW;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < T::NC; ++c) load_words<T::KB>(row + 4 * i * ROW + c * 4 * T::KB, r.k[i] + c * T::KW);
        }
        if constexpr (T::STAGED) {
#pragma unroll
            for (int i = 0; i < T::VN; ++i) {
                int c = i * 64 + lane;
                if (T::CHUNKS % 64) c = min(c, T::CHUNKS - 1);  // lanes without a chunk repeat the last
                const uint32_t t = c / (ROW / 16), piece = c % (ROW / 16), page = t < 16 ? pages.p[0] : pages.p[1];
                r.v[i] = ld16(v + (uint64_t)page * (page_rows * ROW) + (slot + (t & (uint32_t)(ps - 1))) * ROW + piece * 16);
            }
        } else {
            const uint32_t page = g < 2 ? pages.p[0] : pages.p[1];
            const uint8_t *row = v + (uint64_t)page * (page_rows * ROW) + (slot + (8 * g & (ps - 1))) * ROW + m * 16;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int n = 0; n < T::N8; ++n) r.v[j * T::N8 + n] = ld16(row + j * ROW + n * 256);
        }
#pragma unroll
        for (int i = 0; i < T::SN; ++i) {
            int c = i * 64 + lane;
            if (T::SCALES % 64) c = min(c, T::SCALES - 1);
            const bool of_v = c >= T::SCALES / 2;
            const uint32_t blk = (of_v ? c - T::SCALES / 2 : c) / 8, t = 4 * (c % 8), page = t < 16 ? pages.p[0] : pages.p[1];
            r.s[i] = ld4((of_v ? vs : ks) + (uint64_t)page * (page_rows * (D / 32)) + (blk << a.c.page_shift) + slot + (t & (uint32_t)(ps - 1)));
        }
    }

    // What a step works on, read back from LDS.
    struct Parts {
        uint32_t v[8][T::VW];
        u32x2 ks[F == BF16 ? 1 : T::NC], vs[F == BF16 ? 1 : T::NS];
    };
    __device__ __forceinline__ void stage(const T &r, Parts &p) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a wave's LDS accesses are in order: no waits
        if constexpr (T::STAGED) {
#pragma unroll
            for (int i = 0; i < T::VN; ++i) {
                int c = i * 64 + lane;
                if (T::CHUNKS % 64) c = min(c, T::CHUNKS - 1);
                *reinterpret_cast<u32x4 *>(lds + c / (ROW / 16) * T::VROW + c % (ROW / 16) * 16) = r.v[i];
            }
        }
#pragma unroll
        for (int i = 0; i < T::SN; ++i) {
            int c = i * 64 + lane;
            if (T::SCALES % 64) c = min(c, T::SCALES - 1);
            *reinterpret_cast<uint32_t *>(lds + T::SOFF + 4 * c) = r.s[i];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if constexpr (F != BF16) {
            const uint8_t *sc = lds + T::SOFF + 8 * (m / 4), *sv = lds + T::SOFF + D + 8 * g;
#pragma unroll
            for (int c = 0; c < T::NC; ++c) p.ks[c] = ld8(sc + (c * 4 + g) * T::E / 32 * 32);
#pragma unroll
            for (int n = 0; n < T::N8; ++n) p.vs[n] = ld8(sv + (n * 4 + m / 4) * 32);
            if constexpr (T::N4 > 0) p.vs[T::N8] = ld8(sv + (T::N8 * 4 + m / 8) * 32);
            if constexpr (T::N2 > 0) p.vs[T::N8 + T::N4] = ld8(sv + (T::N8 * 4 + T::N4 * 2) * 32);
        }
        if constexpr (T::STAGED) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint8_t *row = lds + (8 * g + j) * T::VROW;
#pragma unroll
                for (int n = 0; n < T::N8; ++n) load_words<kBits<F>>(row + (n * 16 + m) * kBits<F>, p.v[j] + n * T::W8);
                if constexpr (T::N4 > 0)
                    load_words<4 * kBits<F> / 8>(row + (T::N8 * 128 + m * 4) * kBits<F> / 8, p.v[j] + T::N8 * T::W8);
                if constexpr (T::N2 > 0)
                    load_words<2 * kBits<F> / 8>(row + (T::N8 * 128 + T::N4 * 64 + m * 2) * kBits<F> / 8,
                                                 p.v[j] + T::N8 * T::W8 + T::N4 * T::W4);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int n = 0; n < T::N8; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) p.v[j][4 * n + i] = r.v[j * T::N8 + n][i];
        }
    }

    // V of the tokens that the query does not see becomes 0: their weights are
    // 0, and 0 times what lies there must not be NaN.
    __device__ __forceinline__ void clear_unseen(Parts &r, int t0) {
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
    __device__ __forceinline__ void add_segment(const Parts &r, int word, u32x2 vs, bf16x8 p, f32x4 *acc) {
        uint32_t c[8][W / 2];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float sc = F == BF16 ? 1.0f : e8m0_operand(j < 4 ? vs.x : vs.y, j & 3);
            expand<F, W>(r.v[j] + word, sc, c[j]);
        }
#pragma unroll
        for (int t = 0; t < W; ++t)
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(column8<W>(c, t)), p, acc[t], 0, 0, 0);
    }

    __device__ __forceinline__ void step(const T &tile, int t0, const bf16x8 *q, Reference &ref, float &sum, f32x4 *acc) {
        // whole tiles that every query head sees need no mask
        const bool whole = t0 + 31 < sp.len && (t0 >= sp.lo || t0 + 31 < a.sinks);
        Parts r;
        stage(tile, r);
        f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < T::NC; ++c) {
                const u32x2 sk = r.ks[F == BF16 ? 0 : c];
                const float sc = F == BF16 ? 1.0f : e8m0_operand((i ? sk.y : sk.x) >> (8 * (m & 3)));
#pragma unroll
                for (int e = 0; e < T::E / 8; ++e) {
                    uint32_t o[4];
                    expand8<F>(tile.k[i] + c * T::KW + e * (kBits<F> / 4), sc, o);
                    s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(u32x4{o[0], o[1], o[2], o[3]}),
                                                                   q[c * (T::E / 8) + e], s[i], 0, 0, 0);
                }
            }
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s[j / 4][j & 3];
        if (!whole) {
            clear_unseen(r, t0);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = sees(t0 + 8 * g + j) ? x[j] : kNegInf;
        }
        float top = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = __builtin_fmaxf(top, x[j]);
        if (__any(top * ref.unit > ref.at + 8.0f)) {
            top = __builtin_fmaxf(top, __shfl_xor(top, 16));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            const float f = raise(ref, top, a.scale, a.far_unit);
            sum *= f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) acc[t] *= f;
        }
        const float base = ref.at == kNegInf ? 0.0f : ref.at;
        // The weights enter the product with V as bfloat16, off by 2^-8 of each at
        // most; the sum takes them as they are. Against binary64 an output is then
        // off by 1.1 to 1.4 times as much as with binary32 weights, its own rounding
        // included; those would need two products in place of one.
        u32x4 p;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float p0 = exp2_fast(__builtin_fmaf(x[j], ref.unit, -base));
            const float p1 = exp2_fast(__builtin_fmaf(x[j + 1], ref.unit, -base));
            sum += p0 + p1;
            p[j / 2] = pack2(p0, p1);
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
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_decode(DecodeArgs a) {
    using T = Tile<F, D>;
    constexpr int LD = D + 4;  // padded row: 16 heads' writes of one element land in different banks
    __shared__ float s_acc[4][16][LD];
    __shared__ float s_ref[4][16], s_sum[4][16];
    __shared__ __align__(16) uint8_t s_tile[4][T::BYTES > 0 ? T::BYTES : 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // ---- this workgroup's piece
    int b, r, len, piece = 0, pieces = 1;
    if (a.parts == nullptr) {  // one workgroup per pair
        b = blockIdx.x / a.rows;
        r = blockIdx.x % a.rows;
        len = length_of(a.b, b);
    } else {
        int before;  // pieces of a pair of the sequences before
        if (a.first != nullptr) {
            b = count_upto(a.first, a.b.seqs, blockIdx.x / a.rows);
            if (b >= a.b.seqs) return;  // more workgroups than pieces
            before = a.first[b];
            pieces = a.first[b + 1] - before;
            len = length_of(a.b, b);
        } else {
            const Plan p = plan_units(a);
            Chunk c = p.first;
            int s0 = 0;
            before = 0;
            while (blockIdx.x >= (uint32_t)(before + c.all) * a.rows) {
                before += c.all;
                s0 += 64;
                if (s0 >= a.b.seqs) return;
                c = pieces_at(a, s0, length_at(a, s0), p.per);
            }
            const int at = __builtin_ctzll(__ballot(blockIdx.x < (uint32_t)(before + c.upto) * a.rows));
            b = s0 + at;
            len = __builtin_amdgcn_readlane(c.len, at);
            pieces = __builtin_amdgcn_readlane(c.n, at);
            before += __builtin_amdgcn_readlane(c.upto, at) - pieces;
        }
        const uint32_t rest = blockIdx.x - (uint32_t)before * a.rows;
        r = rest / pieces;
        piece = rest % pieces;
        if (piece == 0 && tid == 0) a.found[(int64_t)b * a.rows + r] = int2{(int)blockIdx.x, pieces};
    }

    const int kv_head = __builtin_amdgcn_readfirstlane(r / a.tiles);
    Decoder<F, D> w(a, s_tile[wave], lane, __builtin_amdgcn_readfirstlane(b), kv_head, __builtin_amdgcn_readfirstlane(len));
    const int h0 = r % a.tiles * 16, heads = min(16, a.group - h0);
    const int hq = kv_head * a.group + h0;  // first query head of the pair
    const int u0 = (int)((int64_t)w.sp.n * piece / pieces), u1 = (int)((int64_t)w.sp.n * (piece + 1) / pieces);
    // Q as the right operand, in the element order of K's pieces
    bf16x8 q[D / 32];
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        const int d = (s * 8 / T::E * 4 + w.g) * T::E + s * 8 % T::E;
        u32x4 t = {0, 0, 0, 0};
        if (w.m < heads) t = ld16(a.q + (int64_t)w.b * a.qt + (int64_t)(hq + w.m) * a.qh + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = (t[i] & a.q_keep) ^ a.q_flip;
        q[s] = as_bf16x8(t);
    }
    f32x4 acc[D / 16];
#pragma unroll
    for (int t = 0; t < D / 16; ++t) acc[t] = f32x4{0, 0, 0, 0};
    Reference running = {kNegInf, a.scale};
    float sum = 0.0f;
    T cur, nxt;
    const auto token = [&](int u) { return w.unit_token(u) + 32 * wave; };
    // Two tiles in turn, the next one's loads in flight: issued before the step,
    // which the scheduling barriers keep (it would move them down to their
    // use), and unconditional in the loop, so that the wait for one tile leaves
    // the other's in flight. The last one or two units come after it.
    const auto load = [&](T &r, int u, typename Decoder<F, D>::Pages p) {
        w.load(r, token(u), p);
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto step = [&](const T &r, int u) {
        w.step(r, token(u), q, running, sum, acc);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (u0 < u1) {
        load(cur, u0, w.pages_of(token(u0)));
        auto next = w.pages_of(token(u0 + 1));
        int u = u0;
        for (; u + 2 < u1; u += 2) {
            load(nxt, u + 1, next);
            next = w.pages_of(token(u + 2));
            step(cur, u);
            load(cur, u + 2, next);
            next = w.pages_of(token(u + 3));
            step(nxt, u + 1);
        }
        if (u + 1 < u1) {
            load(nxt, u + 1, next);
            step(cur, u);
            step(nxt, u + 1);
        } else {
            step(cur, u);
        }
    }
    // ---- the four waves' sums meet in LDS
    const float ref = scaled(running, a.scale);
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
    float *part = a.parts + (int64_t)blockIdx.x * (16 * D + 32);
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
        if (pieces == 1) {
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
            const int64_t row = (int64_t)w.b * a.rows / a.tiles * a.group + hq + h;
            *reinterpret_cast<u32x2 *>(a.out + row * D + d) =
                u32x2{pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv)};
            if (d == 0 && a.lse) a.lse[row] = total == 0.0f ? kNegInf : (top + __builtin_amdgcn_logf(total)) * kLn2;
        } else {
            *reinterpret_cast<f32x4 *>(part + h * D + d) = o;
            if (d == 0) {
                part[16 * D + h] = top;
                part[16 * D + 16 + h] = total;
            }
        }
    }
}

// Joins the pieces of each pair, in order. W waves per (sequence, query head):
// one where there are many heads (few of them are split), four where there
// are few (their pieces are many). D / 4 lanes take a piece, and all pieces
// of the first round are loaded before their references are known.
template <int D, int W>
__global__ __launch_bounds__(256) void k_decode_join(DecodeArgs a) {
    constexpr int L = D / 4, PW = 64 / L, SUBS = W * PW, SLOT = 16 * D + 32, R = 4;
    __shared__ float s_o[4 * PW][D];
    __shared__ float s_sum[4 * PW];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kv_heads = a.rows / a.tiles, q_heads = kv_heads * a.group;
    const int64_t row = (int64_t)blockIdx.x * (4 / W) + wave / W;  // sequence, query head
    if (row >= (int64_t)a.b.seqs * q_heads) return;                // W == 1 only: no barrier below
    const int b = (int)(row / q_heads), hq = (int)(row % q_heads);
    const int kv_head = hq / a.group, hg = hq % a.group;
    const int r = kv_head * a.tiles + hg / 16, h = hg % 16;
    const int2 found = a.found[(int64_t)b * a.rows + r];
    const int count = found.y;
    if (count == 1) return;  // written by its workgroup
    const float *part = a.parts + (int64_t)found.x * SLOT;
    const int sub = wave % W * PW + lane / L, d = lane % L * 4;
    const bool on = lane < PW * L;
    const auto at = [&](int k) { return part + (int64_t)(k * SUBS + sub < count ? k * SUBS + sub : 0) * SLOT; };
    f32x4 v[R];
    float vr[R], vs[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        v[k] = *reinterpret_cast<const f32x4 *>(at(k) + h * D + d);
        vr[k] = at(k)[16 * D + h];
        vs[k] = at(k)[16 * D + 16 + h];
    }
    float top = kNegInf;
    for (int i = lane; i < count; i += 64) top = __builtin_fmaxf(top, part[(int64_t)i * SLOT + 16 * D + h]);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, k));
    f32x4 o = {0, 0, 0, 0};
    float sum = 0.0f;
    const auto add = [&](int k, f32x4 x, float ref, float s) {
        if (k * SUBS + sub < count) {
            const float f = ref == top ? 1.0f : exp2_fast(ref - top);
            o += x * f;
            sum += s * f;
        }
    };
#pragma unroll
    for (int k = 0; k < R; ++k) add(k, v[k], vr[k], vs[k]);
    for (int k = R; k * SUBS < count; ++k) {
        const float *p = at(k);
        add(k, *reinterpret_cast<const f32x4 *>(p + h * D + d), p[16 * D + h], p[16 * D + 16 + h]);
    }
    // the W waves' parts meet in LDS
    const int s0 = wave / W * SUBS;
    if (on) {
        *reinterpret_cast<f32x4 *>(&s_o[s0 + sub][d]) = o;
        if (d == 0) s_sum[s0 + sub] = sum;
    }
    if constexpr (W > 1) __syncthreads();
    else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
    if (wave % W != 0 || lane >= L) return;
    o = f32x4{0, 0, 0, 0};
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < SUBS; ++k) {
        o += *reinterpret_cast<const f32x4 *>(&s_o[s0 + k][d]);
        sum += s_sum[s0 + k];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    *reinterpret_cast<u32x2 *>(a.out + row * D + d) = u32x2{pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv)};
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.0f ? kNegInf : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// How the host cuts the work: the most units a sequence can have (from the
// table's width, the window and the sinks), and the number of workgroups.
struct Cut {
    int64_t units, pairs, blocks;
    int tiles;
};

Cut plan_of(const qbn_kv_cache &c, const qbn_kv_batch &b, int q_heads, int window, int sinks) {
    Cut p;
    p.tiles = (q_heads / c.heads + 15) / 16;
    p.pairs = b.seqs * c.heads * p.tiles;
    p.units = (b.row * c.page_size + kUnit - 1) / kUnit;
    if (window > 0) {
        const int64_t seen = (int64_t)window / kUnit + 2 + ((int64_t)sinks + kUnit - 1) / kUnit;
        if (seen < p.units) p.units = seen;
    }
    // Up to two units a pair: one workgroup each. More: as many pieces as run at
    // once (two workgroups of 256 threads on a compute unit, one where the
    // head's sums take more than 256 registers).
    p.blocks = p.units <= 2 ? 0 : c.head_dim <= 128 ? 512 : 256;
    return p;
}

// Pieces at most: a pair of n units has less than n / per + 1, with per at
// least total / blocks; and none has less than one unit.
int64_t most_pieces(const Cut &p) {
    const int64_t most = p.blocks + p.pairs;
    return p.pairs * p.units < most ? p.pairs * p.units : most;
}

// Bytes of the pieces and of the list of where they are, and with the list of
// the sequences' first ones.
int64_t piece_bytes(const Cut &p, int head_dim) { return most_pieces(p) * (16 * (int64_t)head_dim + 32) * 4 + p.pairs * 8; }

template <int F>
hipError_t launch(const DecodeArgs &a, int64_t grid, hipStream_t s) {
    const dim3 g((unsigned)grid);
    if (a.first) k_decode_plan<<<1, kPlanThreads, 0, s>>>(a);
    const int64_t rows = (int64_t)a.b.seqs * a.rows / a.tiles * a.group;
#define QBN_KV_DIM(DD)                                            \
    case DD:                                                      \
        k_decode<F, DD><<<g, 256, 0, s>>>(a);                     \
        if (!a.parts) break;                                      \
        if (rows < 1024) k_decode_join<DD, 4><<<(unsigned)rows, 256, 0, s>>>(a);              \
        else k_decode_join<DD, 1><<<(unsigned)((rows + 3) / 4), 256, 0, s>>>(a);              \
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
    const Cut p = plan_of(c, b, q_heads, window, sinks);
    const int64_t rows = b.seqs * q_heads, joins = rows < 1024 ? rows : (rows + 3) / 4;
    if ((p.blocks ? most_pieces(p) : p.pairs) >= kGridThreads / 256 || (p.blocks && joins >= kGridThreads / 256)) return -1;
    if (p.blocks == 0) return 0;
    return piece_bytes(p, c.head_dim) + (b.seqs > kScanned ? 4 * (b.seqs + 1) : 0);
}

hipError_t launch_kv_decode(const qbn_kv_cache &c, int64_t layer, const qbn_kv_batch &b, int q_heads, const KvRows &q,
                            float scale, int window, int sinks, void *out, float *lse, void *ws, hipStream_t s) {
    const Cut p = plan_of(c, b, q_heads, window, sinks);
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
    a.found = p.blocks ? (int2 *)(a.parts + most_pieces(p) * (16 * c.head_dim + 32)) : nullptr;
    a.first = p.blocks && b.seqs > kScanned ? (int32_t *)((uint8_t *)ws + piece_bytes(p, c.head_dim)) : nullptr;
    a.scale = scale == 0.0f ? 1.0f : fabsf(scale) * kLog2e;
    a.far_unit = ldexpf(1.0f, ilogbf(a.scale));
    a.q_keep = scale == 0.0f ? 0u : ~0u;
    a.q_flip = scale < 0.0f ? 0x80008000u : 0u;
    a.group = q_heads / c.heads, a.tiles = p.tiles, a.rows = c.heads * p.tiles;
    a.window = window, a.sinks = sinks, a.blocks = (int)p.blocks, a.dim = c.head_dim;
    const int64_t grid = p.blocks ? most_pieces(p) : p.pairs;
    if (c.format == QBN_KV_BF16) return launch<BF16>(a, grid, s);
    return c.format == QBN_MXFP8 ? launch<FP8>(a, grid, s) : launch<FP4>(a, grid, s);
}

}  // namespace qbn
