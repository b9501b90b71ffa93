// Turning vectors by their positions (rotary positions), in memory.
//
//   a' = f (a cos t - b sin t),  b' = f (b cos t + a sin t)
// for pairs (a, b) of the first `rot` elements of a head, t = position *
// frequency. Bound by latency for a step's few tokens and by HBM for prompts: each
// element is read and written once. Cosine and sine are computed, 29 instructions a
// pair, once for all heads of a token: a lane has the same 16 elements (eight
// pairs) of every head that it comes to, a wave 64 / (dim / 16) heads at a time. With
// tables of cosines instead a token would read another 4 bytes an element of one head,
// at positions that are not known in advance. Where tokens are few a token's heads are
// spread over waves, each with angles of its own.
//
// 16384 tokens of 40 heads of 128, bf16: 67 us, 5.0 TB/s, a large copy's rate; 16 tokens: 3.3 us,
// of which 2.4 are an empty kernel's.
#include "rope_device.h"
#include "rope_launch.h"

namespace qbn {
namespace {

using namespace rope;

struct Args {
    Rotation r;
    const int32_t *pos;
    const void *x;
    void *out;
    int64_t xt, xh, ot, oh;  // strides in elements
    int64_t units;           // tokens * slices
    int heads, groups, each, slices;  // each: heads that a wave has at a time
    bool keep;               // out is x: what does not turn is there already
};

template <typename T, bool HALF>
__global__ __launch_bounds__(256) void k_rope(Args a) {
    const int lane = threadIdx.x & 63;
    const int group = lane % a.groups, sub = lane / a.groups;
    const Lane16 at = lane16<HALF>(group, a.r.rot);
    const bool on = sub < a.each && (at.turns || !a.keep);
    u32x2 turns[8];
    load_turns(a.r, at.turns ? 8 * group : 0, turns);
    const int64_t waves = (int64_t)gridDim.x * 4;
    for (int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < a.units; u += waves) {
        const int64_t token = kv::div_i64(u, a.slices);
        const int slice = (int)(u - token * a.slices);
        const T *x = (const T *)a.x + token * a.xt;
        T *out = (T *)a.out + token * a.ot;
        float c[8], s[8];
        spin8(turns, a.r.factor, a.pos[token], c, s);
        for (int h = slice * a.each + sub; h < a.heads; h += a.slices * a.each) {
            if (!on) continue;
            const Eight<T> p = load8(x + h * a.xh + at.first), q = load8(x + h * a.xh + at.second);
            float v[8], w[8];
            floats(p, v);
            floats(q, w);
            if (at.turns) turn16<HALF>(v, w, c, s);
            store8(out + h * a.oh + at.first, v);
            store8(out + h * a.oh + at.second, w);
        }
    }
}

}  // namespace

hipError_t launch_rope(const qbn_rotation &r, int64_t tokens, int heads, int dim, const int32_t *positions,
                       const KvRows &x, const KvRowsOut &out, int dtype, hipStream_t s) {
    Args a;
    a.r = {r.turns, r.rot, r.factor};
    a.pos = positions;
    a.x = x.p, a.out = out.p;
    a.xt = x.token_stride, a.xh = x.head_stride, a.ot = out.token_stride, a.oh = out.head_stride;
    a.heads = heads, a.groups = dim / 16, a.each = 64 / a.groups;
    a.keep = x.p == out.p;
    const int passes = (heads + a.each - 1) / a.each;
    const int64_t spread = (8192 + tokens - 1) / tokens;  // waves that run at once: 32 on each of 256 compute units
    a.slices = (int)(spread < passes ? spread : passes);
    a.units = tokens * a.slices;
    const int64_t blocks = (a.units + 3) / 4;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    const bool half = r.layout == QBN_ROPE_HALF;
    if (dtype == QBN_F32) (half ? k_rope<float, true> : k_rope<float, false>)<<<grid, 256, 0, s>>>(a);
    else (half ? k_rope<__bf16, true> : k_rope<__bf16, false>)<<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace qbn
