// Page bookkeeping of the paged key-value cache, on the device: taking,
// forking, freeing and packing pages between two steps without the host
// reading the tables.
//
// Each call is a plan by one workgroup (who gets which page: order matters
// there, so it is prefix sums over the requests and over the pages' reference
// counts, not atomics) and, where pages move, one wide kernel that copies them
// in all layers and writes the tables that follow from it. The plan is bound
// by latency: its scan reads the counts as 64 pages per wave and step, eight
// steps in flight, ranks come from ballots, with one barrier per pass, and what
// the requests look up stays in LDS where it fits. The copies are bound by HBM.
//
// Measured: a turn of 36 sequences in 309 pages (free, fork, reserve, compact) 30
// us of launches; of 120 sequences in 5238 pages 160 us, of which packing moves
// 691 MB in 132 us (5.2 TB/s; a copy of 2 GiB reaches 4.95).
//
// The only atomics are integer sums of reference counts, exchanges of table
// entries being freed, and minima over request indexes: their order does not
// change any result.
#include "kv_device.h"
#include "kv_launch.h"

namespace qbn {
namespace {

using namespace kv;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kNone = 0x7FFFFFFF;

struct Pool {
    int seqs, row, pages, page_shift;
    int32_t *table, *lens, *refs;
};

struct Work {  // in the caller's workspace
    int32_t *owner;         // [seqs] first request that names the slot
    int32_t *first, *have;  // [count] pages taken before a request / the request's pages or length
    int32_t *src, *dst;     // [pages] moves, or dst: the pages taken
    int32_t *map;           // [pages] where each page is after packing
    int32_t *moves;         // [1] number of moves
};

Work work_of(void *ws, int64_t seqs, int64_t count, int64_t pages) {
    Work w;
    w.moves = (int32_t *)ws;
    w.owner = w.moves + 4;
    w.first = w.owner + seqs;
    w.have = w.first + count;
    w.src = w.have + count;
    w.dst = w.src + pages;
    w.map = w.dst + pages;
    return w;
}

__global__ __launch_bounds__(256) void k_copy_pool(Pool in, Pool out) {
    const int64_t n = (int64_t)gridDim.x * 256, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t i = at; i < (int64_t)in.seqs * in.row; i += n) out.table[i] = in.table[i];
    for (int64_t i = at; i < in.seqs; i += n) out.lens[i] = in.lens[i];
    for (int64_t i = at; i < in.pages; i += n) out.refs[i] = in.refs[i];
}

// Counts the pages p in [begin, end) of this wave's share for which take(p, refs[p]).
struct Share {
    int begin, end;
};

__device__ __forceinline__ Share share_of(int pages) {
    const int per = ((pages + kWaves - 1) / kWaves + 63) / 64 * 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = wave * per;  // pages <= 2^20: no overflow
    return {b < pages ? b : pages, b + per < pages ? b + per : pages};
}

// The counts of 512 pages of a share from p on, eight loads in flight; the first
// 512 are kept in registers over a plan's passes.
struct Held {
    int r[8];
};
__device__ __forceinline__ Held hold(const int32_t *refs, Share s, int p) {
    const int lane = threadIdx.x & 63;
    Held h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h.r[i] = p + 64 * i + lane < s.end ? refs[p + 64 * i + lane] : 0;
    return h;
}

template <typename Fn>
__device__ __forceinline__ int count_pages(const int32_t *refs, Share s, const Held &first, Fn take) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int p = s.begin; p < s.end; p += 512) {
        const Held h = p == s.begin ? first : hold(refs, s, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int q = p + 64 * i + lane;
            n += __popcll(__ballot(q < s.end && take(q, h.r[i])));
        }
    }
    return n;
}

// emit(page, rank) for the pages taken, in order; `rank` counts from `base`.
template <typename Fn, typename Out>
__device__ __forceinline__ void list_pages(const int32_t *refs, Share s, const Held &first, int base, Fn take, Out emit) {
    const int lane = threadIdx.x & 63;
    for (int p = s.begin; p < s.end; p += 512) {
        const Held h = p == s.begin ? first : hold(refs, s, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int q = p + 64 * i + lane;
            const bool on = q < s.end && take(q, h.r[i]);
            const uint64_t votes = __ballot(on);
            if (on) emit(q, base + __popcll(votes & ((1ull << lane) - 1)));
            base += __popcll(votes);
        }
    }
}

// Per-wave counts -> the count of the waves before and of all.
__device__ __forceinline__ int wave_prefix(int n, int *lds, int &total) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = n;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += lds[w];
        total += lds[w];
    }
    __syncthreads();
    return before;
}

struct IsFree {
    __device__ bool operator()(int, int refs) const { return refs == 0; }
};

// What a plan's requests look up: in LDS up to these sizes, else in the workspace.
constexpr int kNearSlots = 8192, kNearRequests = 2048, kNearPages = 4096;
struct Near {
    int32_t owner[kNearSlots], first[kNearRequests], pages[kNearPages];
};

// Slots named by requests: owner[slot] = the first request that names it.
__device__ __forceinline__ void claim(const Pool &p, const Work &w, const int32_t *rows, int count) {
    for (int i = threadIdx.x; i < p.seqs; i += kThreads) w.owner[i] = kNone;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads)
        if ((uint32_t)rows[i] < (uint32_t)p.seqs) atomicMin(&w.owner[rows[i]], i);
    __syncthreads();
}

// Takes the pages that the requests need: need(i) pages for request i, or < 0
// if it cannot be met for another reason. Returns true if all can be met
// (then first[i] and the pages dst[0..total) are set, with one reference
// each), else writes the first that cannot to *status.
template <typename Need>
__device__ __forceinline__ bool take_pages(const Pool &p, const Work &w, int count, int32_t *status, Need need, int &total_out,
                                           int32_t *near_pages = nullptr) {
    __shared__ int64_t s_scan[kWaves + 1];
    __shared__ int s_wave[kWaves];
    __shared__ int s_fail;
    const Share sh = share_of(p.pages);
    const Held held = hold(p.refs, sh, sh.begin);
    int free_pages;
    const int before_free = wave_prefix(count_pages(p.refs, sh, held, IsFree{}), s_wave, free_pages);
    if (threadIdx.x == 0) s_fail = kNone;
    const int each = (count + kThreads - 1) / kThreads;
    const int i0 = (int)threadIdx.x * each < count ? (int)threadIdx.x * each : count;
    const int i1 = i0 + each < count ? i0 + each : count;
    int64_t mine = 0, own = 0;  // own: the last request's, which is all of them where each is 1
    int fail = kNone;
    for (int i = i0; i < i1; ++i) {
        own = need(i);
        if (own < 0) fail = i < fail ? i : fail;
        else mine += own;
    }
    int64_t total;
    int64_t at = block_scan<kThreads>(mine, s_scan, total);  // its barriers also order s_fail
    for (int i = i0; i < i1; ++i) {
        const int64_t n = each == 1 ? own : need(i);
        if (n < 0) continue;
        if (n > 0 && at + n > free_pages) fail = i < fail ? i : fail;
        w.first[i] = (int)(at < kNone ? at : kNone);
        at += n;
    }
    if (fail != kNone) atomicMin(&s_fail, fail);
    __syncthreads();
    if (threadIdx.x == 0) *status = s_fail == kNone ? -1 : s_fail;
    if (s_fail != kNone) return false;
    const int t = (int)total;  // <= free_pages
    int32_t *const taken = near_pages && t <= kNearPages ? near_pages : w.dst;
    list_pages(p.refs, sh, held, before_free, IsFree{}, [&](int page, int rank) {
        if (rank < t) {
            taken[rank] = page;
            p.refs[page] = 1;
        }
    });
    total_out = t;
    __syncthreads();
    return true;
}

__global__ __launch_bounds__(kThreads) void k_reserve(Pool p, Work w, int count, const int32_t *rows,
                                                      const int32_t *tokens, int32_t *status) {
    __shared__ Near s_near;
    if (p.seqs <= kNearSlots) w.owner = s_near.owner;
    if (count <= kNearRequests) w.first = s_near.first;
    claim(p, w, rows, count);
    const int ps = 1 << p.page_shift;
    int total = 0;
    const bool ok = take_pages(p, w, count, status, [&](int i) -> int64_t {
        const int s = rows[i], t = tokens[i];
        if ((uint32_t)s >= (uint32_t)p.seqs || w.owner[s] != i || t < 0) return -1;
        const int len = p.lens[s];
        if (len < 0) return -1;
        const int64_t have = ((int64_t)len + ps - 1) >> p.page_shift;
        const int64_t want = ((int64_t)len + t + ps - 1) >> p.page_shift;
        if (want > p.row) return -1;
        return want - have;
    }, total, s_near.pages);
    if (!ok) return;
    const int32_t *const taken = total <= kNearPages ? s_near.pages : w.dst;
    for (int k = threadIdx.x; k < total; k += kThreads) {  // page k goes to the last request whose first is <= k
        int lo = 0, hi = count - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (w.first[mid] <= k) lo = mid;
            else hi = mid - 1;
        }
        const int s = rows[lo];
        const int have = (int)(((int64_t)p.lens[s] + ps - 1) >> p.page_shift);
        p.table[(int64_t)s * p.row + have + (k - w.first[lo])] = taken[k];
    }
    __syncthreads();  // lens are read above
    for (int i = threadIdx.x; i < count; i += kThreads) p.lens[rows[i]] += tokens[i];
}

__global__ __launch_bounds__(kThreads) void k_fork(Pool p, Work w, int count, const int32_t *parents,
                                                   const int32_t *children, int32_t *status) {
    __shared__ int32_t s_owner[kNearSlots];
    if (p.seqs <= kNearSlots) w.owner = s_owner;
    claim(p, w, children, count);
    const int ps = 1 << p.page_shift;
    int total = 0;
    const bool ok = take_pages(p, w, count, status, [&](int i) -> int64_t {
        const int a = parents[i], c = children[i];
        if ((uint32_t)a >= (uint32_t)p.seqs || (uint32_t)c >= (uint32_t)p.seqs || a == c || w.owner[c] != i) return -1;
        const int len = p.lens[a];
        if (p.lens[c] != 0 || len < 0 || (((int64_t)len + ps - 1) >> p.page_shift) > p.row) return -1;
        if ((len & (ps - 1)) == 0) return 0;
        if ((uint32_t)p.table[(int64_t)a * p.row + (len >> p.page_shift)] >= (uint32_t)p.pages) return -1;
        return 1;
    }, total);
    if (threadIdx.x == 0) *w.moves = ok ? total : 0;
    if (!ok) return;
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const int a = parents[i], len = p.lens[a];
        w.have[i] = len;
        if (len & (ps - 1)) w.src[w.first[i]] = p.table[(int64_t)a * p.row + (len >> p.page_shift)];
    }
}

// The entries of the children's rows, spread over the grid: whole pages shared,
// the copied page, then none.
__device__ __forceinline__ void fork_rows(const Pool &p, const Work &w, int count, const int32_t *parents, const int32_t *children) {
    const int64_t n = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)count * p.row; i += n) {
        const int r = (int)(i / p.row), j = (int)(i % p.row);
        const int a = parents[r], c = children[r], len = w.have[r];
        const int full = len >> p.page_shift;
        int e = -1;
        if (j < full) {
            e = p.table[(int64_t)a * p.row + j];
            if ((uint32_t)e < (uint32_t)p.pages) atomicAdd(&p.refs[e], 1);
        } else if (j == full && (len & ((1 << p.page_shift) - 1))) {
            e = w.dst[w.first[r]];
        }
        p.table[(int64_t)c * p.row + j] = e;
        if (j == 0) p.lens[c] = len;
    }
}

__global__ __launch_bounds__(256) void k_free(Pool p, int count, const int32_t *rows, int window, int sinks) {
    for (int r = blockIdx.y; r < count; r += gridDim.y) {
        const int s = rows[r];
        if ((uint32_t)s >= (uint32_t)p.seqs) continue;
        int j0 = 0, j1 = p.row;
        if (window > 0) {
            const int64_t end = (int64_t)p.lens[s] - window;  // tokens before it are out of the window
            j0 = (int)(((int64_t)sinks + (1 << p.page_shift) - 1) >> p.page_shift < p.row
                           ? ((int64_t)sinks + (1 << p.page_shift) - 1) >> p.page_shift
                           : p.row);
            const int64_t e = end > 0 ? end >> p.page_shift : 0;
            j1 = (int)(e < p.row ? e : p.row);
        }
        for (int j = j0 + blockIdx.x * 256 + threadIdx.x; j < j1; j += gridDim.x * 256) {
            const int e = atomicExch(&p.table[(int64_t)s * p.row + j], -1);
            if ((uint32_t)e < (uint32_t)p.pages) atomicSub(&p.refs[e], 1);
        }
        if (window <= 0 && blockIdx.x == 0 && threadIdx.x == 0) p.lens[s] = 0;
    }
}

// Both in one workgroup, for tables that it passes over faster than two kernels
// start: out = in without the pages of the rows named. In one and in two, us:
// 800 entries 2.5 and 4.3, 2040 3.0 and 4.4, 3000 3.5 and 4.4, 4100 4.6 and 4.5,
// 8000 6.5 and 4.4, 15000 10.7 and 4.5.
constexpr int64_t kFreeTable = 4096, kFreePages = 4096;
constexpr int kFreeSlots = 4096;
__global__ __launch_bounds__(kThreads) void k_copy_free(Pool in, Pool out, int count, const int32_t *rows, int window, int sinks) {
    __shared__ uint32_t s_named[kFreeSlots / 32];
    for (int i = threadIdx.x; i < (in.seqs + 31) / 32; i += kThreads) s_named[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads)
        if ((uint32_t)rows[i] < (uint32_t)in.seqs) atomicOr(&s_named[rows[i] / 32], 1u << (rows[i] % 32));
    for (int q = threadIdx.x; q < in.pages; q += kThreads) out.refs[q] = in.refs[q];
    __syncthreads();
    const int first = (int)(((int64_t)sinks + (1 << in.page_shift) - 1) >> in.page_shift < in.row
                                ? ((int64_t)sinks + (1 << in.page_shift) - 1) >> in.page_shift
                                : in.row);
    const int entries = in.seqs * in.row;
    for (int i0 = threadIdx.x; i0 < entries; i0 += 4 * kThreads) {
        int e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = i0 + k * kThreads < entries ? in.table[i0 + k * kThreads] : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= entries) break;
            const int s = i / in.row, j = i % in.row;
            bool gone = s_named[s / 32] >> (s % 32) & 1;
            if (gone && window > 0) {
                const int64_t end = (int64_t)in.lens[s] - window;  // tokens before it are out of the window
                gone = j >= first && j < (end > 0 ? end >> in.page_shift : 0);
            }
            if (gone && (uint32_t)e[k] < (uint32_t)in.pages) atomicSub(&out.refs[e[k]], 1);
            out.table[i] = gone ? -1 : e[k];
        }
    }
    for (int s = threadIdx.x; s < in.seqs; s += kThreads)
        out.lens[s] = window <= 0 && (s_named[s / 32] >> (s % 32) & 1) ? 0 : in.lens[s];
}

__global__ __launch_bounds__(kThreads) void k_compact(Pool p, Work w, int32_t *live_out) {
    __shared__ int s_wave[kWaves];
    const Share sh = share_of(p.pages);
    int live, low;
    const auto used = [](int, int r) { return r > 0; };
    const Held held = hold(p.refs, sh, sh.begin);
    const int before = wave_prefix(count_pages(p.refs, sh, held, used), s_wave, live);
    wave_prefix(count_pages(p.refs, sh, held, [&](int q, int r) { return r > 0 && q < live; }), s_wave, low);
    const int moves = live - low;
    // pages in use, ranked: the ones at or beyond `live` come after the `low` ones below
    list_pages(p.refs, sh, held, before, used, [&](int q, int rank) {
        if (q >= live) w.src[rank - low] = q;
    });
    list_pages(p.refs, sh, held, sh.begin - before, [](int, int r) { return r <= 0; }, [&](int q, int rank) {
        if (q < live) w.dst[rank] = q;
        else w.map[q] = q;  // a broken table may name it: the entry stays
    });
    if (threadIdx.x == 0) {
        *w.moves = moves;
        *live_out = live;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < moves; k += kThreads) {
        const int a = w.src[k], b = w.dst[k];
        w.map[a] = b;
        p.refs[b] = p.refs[a];
        p.refs[a] = 0;
    }
}

struct MoveArgs {
    uint8_t *buf[4];
    int64_t page_bytes[4];   // of one page of one layer
    int64_t layer_bytes[4];
    int layers, bufs;
    int chunks[4], chunk_sum;  // 16 KB pieces of a page in each buffer
};

// Copies pages src[i] -> dst[i] in every layer (the two lists have no page in
// common), and writes the table: the forked rows, or, after packing, the new
// places of the pages at and beyond *word, the number of pages in use.
template <bool FORK>
__global__ __launch_bounds__(256) void k_move(MoveArgs m, Pool p, Work w, int count, const int32_t *parents,
                                              const int32_t *children, const int32_t *word) {
    if constexpr (FORK) {
        if (*word >= 0) return;  // a request could not be met
        fork_rows(p, w, count, parents, children);
    } else {
        const int live = *word;
        const int64_t n = (int64_t)gridDim.x * 256;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)p.seqs * p.row; i += n) {
            const int e = p.table[i];
            if (e >= live && e < p.pages) p.table[i] = w.map[e];
        }
    }
    const int64_t units = (int64_t)*w.moves * m.layers * m.chunk_sum;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t pl = div_i64(u, m.chunk_sum);
        int c = (int)(u - pl * m.chunk_sum);
        const int i = (int)div_i64(pl, m.layers), layer = (int)(pl - (int64_t)i * m.layers);
        int b = 0;
        while (c >= m.chunks[b]) c -= m.chunks[b++];
        const int64_t bytes = m.page_bytes[b], o = (int64_t)c * 16384 + threadIdx.x * 16;
        const uint8_t *src = m.buf[b] + layer * m.layer_bytes[b] + w.src[i] * bytes + o;
        uint8_t *dst = m.buf[b] + layer * m.layer_bytes[b] + w.dst[i] * bytes + o;
        u32x4 t[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (o + k * 4096 < bytes) t[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(src + k * 4096));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (o + k * 4096 < bytes) __builtin_nontemporal_store(t[k], reinterpret_cast<u32x4 *>(dst + k * 4096));
    }
}

MoveArgs move_args(const qbn_kv_cache &c) {
    MoveArgs m;
    const int64_t elems = (int64_t)c.heads * c.page_size * c.head_dim;
    const int bits = c.format == QBN_KV_BF16 ? 16 : c.format == QBN_MXFP8 ? 8 : 4;
    void *buf[4] = {c.k, c.v, c.k_scales, c.v_scales};
    m.layers = (int)c.layers;
    m.bufs = c.format == QBN_KV_BF16 ? 2 : 4;
    m.chunk_sum = 0;
    for (int i = 0; i < 4; ++i) {
        m.buf[i] = (uint8_t *)buf[i];
        m.page_bytes[i] = i < 2 ? elems * bits / 8 : elems / 32;
        m.layer_bytes[i] = m.page_bytes[i] * c.pages;
        m.chunks[i] = i < m.bufs ? (int)((m.page_bytes[i] + 16383) / 16384) : 0;
        m.chunk_sum += m.chunks[i];
    }
    return m;
}

Pool pool_of(const qbn_kv_pool &p) {
    return {(int)p.seqs, (int)p.row, (int)p.pages, __builtin_ctz(p.page_size), p.table, p.lens, p.refs};
}

// All three, since the pointer of a tensor without elements is null.
bool same(const qbn_kv_pool &a, const qbn_kv_pool &b) { return a.table == b.table && a.lens == b.lens && a.refs == b.refs; }

// out = in, where they are not the same tables.
void copy_pool(const qbn_kv_pool &in, const qbn_kv_pool &out, hipStream_t s) {
    if (same(in, out)) return;
    const int64_t most = in.seqs * in.row > in.pages ? in.seqs * in.row : in.pages;
    const int64_t blocks = (most + 255) / 256;
    if (most > 0 || in.seqs > 0)
        k_copy_pool<<<(unsigned)(blocks < 1 ? 1 : blocks < 2048 ? blocks : 2048), 256, 0, s>>>(pool_of(in), pool_of(out));
}

unsigned row_blocks(int64_t row) { return (unsigned)(row < 256 * 64 ? (row + 255) / 256 : 64); }
unsigned at_most(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

}  // namespace

int64_t kv_pool_workspace(const qbn_kv_pool &p, int64_t count) { return 4 * (4 + p.seqs + 2 * count + 3 * p.pages); }

hipError_t launch_kv_reserve(const qbn_kv_pool &in, const qbn_kv_pool &out, int64_t count, const int32_t *rows,
                             const int32_t *tokens, int32_t *status, void *ws, hipStream_t s) {
    copy_pool(in, out, s);
    k_reserve<<<1, kThreads, 0, s>>>(pool_of(out), work_of(ws, out.seqs, count, out.pages), (int)count, rows, tokens, status);
    return hipGetLastError();
}

hipError_t launch_kv_fork(const qbn_kv_cache &c, const qbn_kv_pool &in, const qbn_kv_pool &out, int64_t count,
                          const int32_t *parents, const int32_t *children, int32_t *status, void *ws, hipStream_t s) {
    copy_pool(in, out, s);
    const Pool p = pool_of(out);
    const Work w = work_of(ws, out.seqs, count, out.pages);
    k_fork<<<1, kThreads, 0, s>>>(p, w, (int)count, parents, children, status);
    if (count > 0 && p.row > 0) {
        const MoveArgs m = move_args(c);
        const int64_t copies = count * m.layers * m.chunk_sum, entries = (count * p.row + 255) / 256;
        k_move<true><<<at_most(copies > entries ? copies : entries, 4096), 256, 0, s>>>(m, p, w, (int)count, parents, children, status);
    }
    return hipGetLastError();
}

hipError_t launch_kv_free(const qbn_kv_pool &in, const qbn_kv_pool &out, int64_t count, const int32_t *rows,
                          int window, int sinks, hipStream_t s) {
    if (!same(in, out) && in.seqs * in.row <= kFreeTable && in.pages <= kFreePages && in.seqs <= kFreeSlots && count <= kFreeSlots) {
        k_copy_free<<<1, kThreads, 0, s>>>(pool_of(in), pool_of(out), (int)count, rows, window, sinks);
        return hipGetLastError();
    }
    copy_pool(in, out, s);
    if (count > 0)
        k_free<<<dim3(out.row > 0 ? row_blocks(out.row) : 1, at_most(count, 4096)), 256, 0, s>>>(pool_of(out), (int)count, rows, window, sinks);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const qbn_kv_cache &c, const qbn_kv_pool &in, const qbn_kv_pool &out, int32_t *live,
                             void *ws, hipStream_t s) {
    copy_pool(in, out, s);
    const Pool p = pool_of(out);
    const Work w = work_of(ws, out.seqs, 0, out.pages);
    k_compact<<<1, kThreads, 0, s>>>(p, w, live);
    const MoveArgs m = move_args(c);
    k_move<false><<<4096, 256, 0, s>>>(m, p, w, 0, nullptr, nullptr, live);
    return hipGetLastError();
}

}  // namespace qbn
