// Rotation of q and k by positions on several axes, without a cache:
//     (a, b) -> bf16(a cos - b sin), bf16(b cos + a sin)
// of a pair's two values, with the row of the tables that the token's position
// on the pair's axis names.  Each product is rounded and then the sum, as in the
// append (kv4_append.cu), so both give the same bits.
//
// Memory bound.  A lane takes eight pairs, both sides (two 16-byte steps), of heads one
// after the other, with their cosines and sines in registers; a warp has one
// token, so positions and tables are looked up once for all its heads, while
// the first ones are on their way (rope_heads()).
//
// Measured: 32 + 8 heads of 128, 8143 tokens 28.8 us (5.9 TB/s, 0.86 of a copy): with two heads a lane
// on their way and 64 registers a thread; with one 31, with three 30, with three CTAs an SM instead of four 32,
// with warps of 8 rounds instead of all heads 31.  16 + 16 heads of 64, 8620 tokens (in L2) 10.9 us; one token 2.1
// (32 + 8 heads of 128 on three axes 2.4).
#include "kernels.h"
#include "kv4_host.h"
#include "rope.cuh"

namespace uw {

namespace {

struct RopeParams {
    Rows q, k, qo, ko;
    Axes axes;
    RopePlan plan;
    const float *cos, *sin;
    int64_t n_tokens, rope_len;
    int32_t q_heads, heads;           // of q, and of q and k
    float minus_zero;                 // -0, which the compiler does not know (rotate())
    uint32_t *status;
};

template <bool kInterleaved>
__global__ void __launch_bounds__(256, 4) rope_kernel(const RopeParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const uint64_t unit = uint64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const uint32_t units = uint32_t(p.plan.units);
    const int64_t t = (unit >> 32) ? unit / units : uint32_t(unit) / units;
    if (t >= p.n_tokens)
        return;
    const int first = int(unit - uint64_t(t) * units) * p.plan.rounds * p.plan.per;  // the warp's first head
    auto at = [&](const Rows &q, const Rows &k, int j) {
        const bool is_k = j >= p.q_heads;
        const Rows &rows = is_k ? k : q;
        return rows.p + t * rows.ts + (is_k ? j - p.q_heads : j) * rows.hs;
    };
    rope_heads<kInterleaved>(
        p.plan, p.axes, p.cos, p.sin, pair2(p.minus_zero, p.minus_zero), first, p.heads,
        [&](int j) { return at(p.q, p.k, j); }, [&](int j) { return at(p.qo, p.ko, j); },
        [&](AxesAt &turn) {
            if (turn.find(p.axes, t, p.rope_len))
                return true;
            if ((threadIdx.x & 31) == 0)
                atomicOr(p.status, kStatusBadCache);
            return false;
        });
}

}  // namespace

uw_status rope_axes_map(const uw_rope &r, int64_t n_tokens, Axes *a) {
    if (r.rot_dim == 0) {  // nothing turns: positions and axes are not looked at
        *a = Axes{};
        return UW_OK;
    }
    if (r.n_axes < 1 || r.axis_stride < 0 || (n_tokens > 0 && !r.pos_dev) || !r.pair_axis ||
        (reinterpret_cast<uintptr_t>(r.pos_dev) & 3) || (r.n_axes > 1 && r.axis_stride != 0 && r.axis_stride < n_tokens))
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
    p.plan = RopePlan(n_tokens, p.heads, r->rot_dim, head_dim, 2 * 4 * int64_t(sm_count()));
    p.minus_zero = -0.f;
    p.status = static_cast<uint32_t *>(ws);
    const int64_t units = n_tokens * p.plan.units;
    if (units > int64_t(8) * 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    const dim3 grid(unsigned((units + 7) / 8));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (r->interleaved ? launch_overlapped(rope_kernel<true>, grid, dim3(256), 0, st, p)
                           : launch_overlapped(rope_kernel<false>, grid, dim3(256), 0, st, p)) == cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}
