// Rotation of q and k by positions on several axes, without a cache:
//     (a, b) -> bf16(a cos - b sin), bf16(b cos + a sin)
// of a pair's two values, with the row of the tables that the token's position
// on the pair's axis names.  Each product is rounded and then the sum, as in the
// append (kv4_append.cu), so both give the same bits.
//
// Memory bound.  A lane takes eight pairs, both sides (two 16-byte steps), of heads one
// after the other, with their cosines and sines in registers; a warp has one
// token, so positions and tables are looked up once for all its heads, while
// the first ones are on their way.  A lane reads what it writes, so q_out
// may be q.
#include "kernels.h"
#include "kv4_host.h"
#include "rope.cuh"

namespace uw {

namespace {

struct RopeParams {
    Rows q, k, qo, ko;
    Axes axes;
    const float *cos, *sin;
    int64_t n_tokens, rope_len;
    int32_t q_heads, heads;           // of q, and of q and k
    int32_t half;                     // pairs
    int32_t lanes, per;               // of a head, and heads a warp takes at once
    int32_t rounds, units;            // heads a lane takes one after the other; warps a token
    int32_t tail;                     // 16-byte steps of a head that are not rotated
    bool copy_q, copy_k;              // and are to be copied
    float minus_zero;                 // -0, which the compiler does not know (rotate())
    uint32_t *status;
};

constexpr int kAhead = 2;  // heads a lane has on their way

template <bool kInterleaved>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const uint64_t unit = uint64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = (unit >> 32) ? unit / uint32_t(p.units) : uint32_t(unit) / uint32_t(p.units);
    if (t >= p.n_tokens)
        return;
    const int first = int(unit - uint64_t(t) * p.units) * p.rounds * p.per;  // the warp's first head
    const int mine = lane / p.lanes, pc = lane - mine * p.lanes;
    const bool busy = mine < p.per;
    const int at0 = kInterleaved ? 16 * pc : 8 * pc, at1 = kInterleaved ? at0 + 8 : p.half + at0;
    uint4 x[kAhead][2];
    auto fetch = [&](int n0) {
#pragma unroll
        for (int n = 0; n < kAhead; n++) {
            const int j = first + (n0 + n) * p.per + mine;
            const bool in = busy && n0 + n < p.rounds && j < p.heads, is_k = j >= p.q_heads;
            const Rows &src = is_k ? p.k : p.q;
            const uint16_t *const at = src.p + t * src.ts + (is_k ? j - p.q_heads : j) * src.hs;
            x[n][0] = in ? *reinterpret_cast<const uint4 *>(at + at0) : make_uint4(0, 0, 0, 0);
            x[n][1] = in ? *reinterpret_cast<const uint4 *>(at + at1) : make_uint4(0, 0, 0, 0);
        }
    };
    fetch(0);
    AxesAt turn;
    if (!turn.find(p.axes, t, p.rope_len)) {
        if (lane == 0)
            atomicOr(p.status, kStatusBadCache);
        return;
    }
    Rotation r[2];
    r[0].on = r[1].on = true;
    r[0].interleaved = r[1].interleaved = kInterleaved;
    if (busy) {
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const float4 cs = turn.four(p.axes, p.cos, p.half, 8 * pc + 4 * k);
            const float4 sn = turn.four(p.axes, p.sin, p.half, 8 * pc + 4 * k);
            if (kInterleaved) {
                r[k].of_pairs(cs, sn);
            } else {
                r[0].of_side(cs, sn, k, false);
                r[1].of_side(cs, sn, k, true);
            }
        }
    }
    const uint64_t zero = pair2(p.minus_zero, p.minus_zero);
    for (int n0 = 0; n0 < p.rounds;) {
#pragma unroll
        for (int n = 0; n < kAhead; n++) {
            const int j = first + (n0 + n) * p.per + mine;
            uint32_t a[4] = {x[n][0].x, x[n][0].y, x[n][0].z, x[n][0].w};
            uint32_t b[4] = {x[n][1].x, x[n][1].y, x[n][1].z, x[n][1].w};
            rotate(r[0], zero, a, x[n][1]);
            rotate(r[1], zero, b, x[n][0]);
            if (busy && n0 + n < p.rounds && j < p.heads) {
                const bool is_k = j >= p.q_heads;
                const Rows &dst = is_k ? p.ko : p.qo;
                uint16_t *const at = dst.p + t * dst.ts + (is_k ? j - p.q_heads : j) * dst.hs;
                *reinterpret_cast<uint4 *>(at + at0) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4 *>(at + at1) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        }
        n0 += kAhead;
        if (n0 < p.rounds)
            fetch(n0);
    }
    if (!p.tail)
        return;
    const int last = min(first + p.rounds * p.per, p.heads);
    for (int i = lane; i < (last - first) * p.tail; i += 32) {
        const int j = first + i / p.tail, at = 2 * p.half + 8 * (i % p.tail);
        const bool is_k = j >= p.q_heads;
        if (!(is_k ? p.copy_k : p.copy_q))
            continue;
        const Rows &src = is_k ? p.k : p.q, &dst = is_k ? p.ko : p.qo;
        const int h = is_k ? j - p.q_heads : j;
        *reinterpret_cast<uint4 *>(dst.p + t * dst.ts + h * dst.hs + at) =
            *reinterpret_cast<const uint4 *>(src.p + t * src.ts + h * src.hs + at);
    }
}

}  // namespace

uw_status rope_axes_map(const uw_rope &r, int64_t n_tokens, Axes *a) {
    if (r.n_axes < 1 || r.axis_stride < 0 || (n_tokens > 0 && !r.pos_dev) || (r.rot_dim > 0 && !r.pair_axis) ||
        (reinterpret_cast<uintptr_t>(r.pos_dev) & 3) || (r.n_axes > 1 && r.axis_stride < n_tokens))
        return UW_ERR_INVALID_ARG;
    if (r.n_axes > kMaxAxes || r.rot_dim > 2 * kMaxPairs)
        return UW_ERR_UNSUPPORTED;
    *a = Axes{r.pos_dev, r.axis_stride, r.n_axes, {}};
    for (int i = 0; i < r.rot_dim / 2; i++) {
        if (r.pair_axis[i] >= r.n_axes)
            return UW_ERR_INVALID_ARG;
        a->map[i / 16] |= uint32_t(r.pair_axis[i]) << (2 * (i % 16));
    }
    return UW_OK;
}

}  // namespace uw

using namespace uw;

extern "C" uw_status uw_rope_axes(const uw_rope *r, int64_t n_tokens, const uw_kv4_rows *q, int32_t q_heads,
                                  const uw_kv4_rows *q_out, const uw_kv4_rows *k, int32_t k_heads,
                                  const uw_kv4_rows *k_out, int32_t head_dim, void *ws, size_t ws_bytes,
                                  void *stream) {
    if (!r || n_tokens < 0 || q_heads < 0 || k_heads < 0 || (q_heads > 0) != (q != nullptr) ||
        (q_heads > 0) != (q_out != nullptr) || (k_heads > 0) != (k != nullptr) || (k_heads > 0) != (k_out != nullptr) ||
        r->rot_dim < 0 || r->rope_len < 0 || !r->cos_dev || !r->sin_dev || !ws)
        return UW_ERR_INVALID_ARG;
    if (head_dim <= 0 || q_heads + int64_t(k_heads) == 0)
        return UW_ERR_SHAPE;
    if (head_dim % 8 || r->rot_dim == 0 || r->rot_dim % 16 || r->rot_dim > head_dim || head_dim > 0x10000 ||
        q_heads > kKv4MaxHeads || k_heads > kKv4MaxHeads || n_tokens > 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    if (((reinterpret_cast<uintptr_t>(r->cos_dev) | reinterpret_cast<uintptr_t>(r->sin_dev)) & 15) ||
        (reinterpret_cast<uintptr_t>(ws) & 255))
        return UW_ERR_INVALID_ARG;
    if (ws_bytes < 256)
        return UW_ERR_BUFFER_TOO_SMALL;
    RopeParams p{};
    const uw_status s = rope_axes_map(*r, n_tokens, &p.axes);
    if (s != UW_OK || n_tokens == 0)
        return s;
    if ((q && (!kv4_rows(q, &p.q) || !kv4_rows(q_out, &p.qo))) || (k && (!kv4_rows(k, &p.k) || !kv4_rows(k_out, &p.ko))))
        return UW_ERR_INVALID_ARG;
    p.cos = r->cos_dev;
    p.sin = r->sin_dev;
    p.n_tokens = n_tokens;
    p.rope_len = r->rope_len;
    p.q_heads = q_heads;
    p.heads = q_heads + k_heads;
    p.half = r->rot_dim / 2;
    p.lanes = r->rot_dim / 16;
    p.per = 32 / p.lanes;
    p.tail = (head_dim - r->rot_dim) / 8;
    auto moved = [](const Rows &a, const Rows &b) { return a.p != b.p || a.ts != b.ts || a.hs != b.hs; };
    p.copy_q = moved(p.q, p.qo);
    p.copy_k = moved(p.k, p.ko);
    p.minus_zero = -0.f;
    p.status = static_cast<uint32_t *>(ws);
    const int all = (p.heads + p.per - 1) / p.per;
    // warps for two per scheduler come first, longer ones after that
    const int64_t two = 2 * 4 * int64_t(sm_count());
    p.rounds = 1;
    while (2 * p.rounds <= 16 && p.rounds < all && n_tokens * ((all + 2 * p.rounds - 1) / (2 * p.rounds)) >= two)
        p.rounds *= 2;
    p.units = (all + p.rounds - 1) / p.rounds;
    const int64_t units = n_tokens * p.units;
    if (units > int64_t(8) * 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    const dim3 grid(unsigned((units + 7) / 8));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (r->interleaved ? launch_overlapped(rope_kernel<true>, grid, dim3(256), 0, st, p)
                           : launch_overlapped(rope_kernel<false>, grid, dim3(256), 0, st, p)) == cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}
