// Attention over the 4-bit paged cache, one warp for each (token, query head):
// the keys one after the other with the running maximum and sum of their
// softmax.  A lane holds D / 32 dimensions.
#include <cmath>

#include "kernels.h"
#include "kv4.cuh"
#include "kv4_host.h"

namespace uw {

uw_status kv4_view(const uw_kv4_cache *c, const int32_t *start, const int32_t *len, int64_t n_tokens, void *ws,
                   size_t ws_bytes, Kv4View *v) {
    // nothing to do needs no buffers (those of empty tensors are null)
    const bool none = n_tokens == 0 || (c && c->n_seqs == 0);
    if (!c || (!none && (!c->pages_dev || !c->table_dev || !start || !len)) || !ws || n_tokens < 0 || c->n_seqs < 0 ||
        c->table_width < 0 || c->table_stride < 0 || c->n_pages < 0 ||
        (c->n_seqs > 1 && c->table_stride < c->table_width))
        return UW_ERR_INVALID_ARG;
    if (c->kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0)
        return UW_ERR_SHAPE;
    if ((c->head_dim != 64 && c->head_dim != 128) || c->page_size < 16 || c->page_size > 256 ||
        (c->page_size & (c->page_size - 1)) || c->kv_heads > kKv4MaxHeads || n_tokens > 0x7fffffff ||
        c->n_pages > 0x7fffffff || int64_t(c->table_width) * c->page_size > 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(c->pages_dev) & 15) ||
        ((reinterpret_cast<uintptr_t>(c->table_dev) | reinterpret_cast<uintptr_t>(start) |
          reinterpret_cast<uintptr_t>(len)) & 3) ||
        (reinterpret_cast<uintptr_t>(ws) & 255))
        return UW_ERR_INVALID_ARG;
    if (ws_bytes < 256)
        return UW_ERR_BUFFER_TOO_SMALL;
    int log2 = 4;
    while ((1 << log2) < c->page_size)
        log2++;
    *v = Kv4View{static_cast<uint8_t *>(c->pages_dev), c->table_dev, c->n_pages, c->table_stride, start, len,
                 none ? 0 : n_tokens,
                 c->table_width, c->n_seqs, c->kv_heads, log2, static_cast<uint32_t *>(ws)};
    return UW_OK;
}

bool kv4_rows(const uw_kv4_rows *r, Rows *out) {
    if (!r->dev || (reinterpret_cast<uintptr_t>(r->dev) & 15) || r->token_stride % 8 || r->head_stride % 8 ||
        r->token_stride < 0 || r->head_stride < 0)
        return false;
    *out = Rows{r->dev, r->token_stride, r->head_stride};
    return true;
}

namespace {

struct AttnParams {
    Kv4View v;
    Rows q, o;
    float *lse;
    float scale;
    int32_t q_heads, group, causal, window;
};

template <int D>
__global__ void __launch_bounds__(256) kv4_attn_kernel(const AttnParams p) {
    constexpr int N = D / 32;  // dimensions a lane
    grid_dep_launch();
    grid_dep_wait();
    const Kv4View &v = p.v;
    const int lane = threadIdx.x & 31;
    const int64_t unit = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = unit / p.q_heads;
    const int h = int(unit - t * p.q_heads);
    if (t >= v.n_tokens)
        return;
    const int s = kv4_find_seq(v, int(t));
    const Seq sq = kv4_seq(v, s);
    if (t < sq.t0 || t >= int64_t(sq.t0) + sq.n)
        return;
    const int32_t pos = sq.len - sq.n + (int32_t(t) - sq.t0);
    const int32_t hi = p.causal ? pos + 1 : sq.len;
    const int32_t lo = p.window ? max(0, pos - p.window + 1) : 0;
    const int hk = h / p.group;
    float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; i++) {
        q[i] = p.scale * bf16_lo(p.q.p[t * p.q.ts + h * p.q.hs + N * lane + i]);
        o[i] = 0.f;
    }
    for (int32_t j = lo; j < hi; j++) {
        const uint8_t *blk = kv4_block<D>(v, s, j, hk);
        if (!blk)
            continue;
        const int slot = j & ((1 << v.page_log2) - 1);
        auto load = [&](int is_v, float (&x)[N]) {
            const uint8_t *row = blk + kv4_codes<D>(v.page_log2, slot, is_v) + N / 2 * lane;
            const uint32_t par = *reinterpret_cast<const uint32_t *>(blk + kv4_params<D>(v.page_log2, slot, is_v));
#pragma unroll
            for (int i = 0; i < N; i++)
                x[i] = fmaf(float((row[i / 2] >> (4 * (i & 1))) & 15), bf16_lo(par), bf16_hi(par));
        };
        float x[N], d = 0.f;
        load(0, x);
#pragma unroll
        for (int i = 0; i < N; i++)
            d = fmaf(q[i], x[i], d);
#pragma unroll
        for (int b = 16; b; b >>= 1)
            d += __shfl_xor_sync(0xffffffffu, d, b);
        const float m2 = fmaxf(m, d), old = m2 == -INFINITY ? 1.f : expf(m - m2);
        const float e = d == -INFINITY ? 0.f : expf(d - m2);
        load(1, x);
        l = l * old + e;
#pragma unroll
        for (int i = 0; i < N; i++)
            o[i] = o[i] * old + e * x[i];
        m = m2;
    }
#pragma unroll
    for (int i = 0; i < N; i++)
        p.o.p[t * p.o.ts + h * p.o.hs + N * lane + i] =
            __bfloat16_as_ushort(__float2bfloat16_rn(l == 0.f ? 0.f : o[i] / l));
    if (p.lse && lane == 0)
        p.lse[t * p.q_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace uw

using namespace uw;

extern "C" uw_status uw_kv4_page_bytes(int32_t kv_heads, int32_t head_dim, int32_t page_size, size_t *bytes) {
    if (!bytes)
        return UW_ERR_INVALID_ARG;
    if (kv_heads <= 0 || head_dim <= 0 || page_size <= 0)
        return UW_ERR_SHAPE;
    if ((head_dim != 64 && head_dim != 128) || page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) ||
        kv_heads > kKv4MaxHeads)
        return UW_ERR_UNSUPPORTED;
    *bytes = size_t(kv_heads) * page_size * (head_dim + 8);
    return UW_OK;
}

extern "C" uw_status uw_kv4_workspace_size(const uw_kv4_cache *c, int32_t q_heads, size_t *bytes) {
    if (!c || !bytes)
        return UW_ERR_INVALID_ARG;
    if (q_heads <= 0 || c->kv_heads <= 0 || q_heads % c->kv_heads)
        return UW_ERR_SHAPE;
    *bytes = 256;
    return UW_OK;
}

extern "C" uw_status uw_kv4_attention(const uw_kv4_cache *c, const int32_t *start, const int32_t *len,
                                      int64_t n_tokens, const uw_kv4_rows *q, int32_t q_heads, const uw_kv4_rows *out,
                                      float *lse, int64_t max_new, int64_t max_len, float softmax_scale,
                                      int32_t causal, int32_t window, void *ws, size_t ws_bytes, void *stream) {
    AttnParams p{};
    const uw_status s = kv4_view(c, start, len, n_tokens, ws, ws_bytes, &p.v);
    if (s != UW_OK)
        return s;
    const bool none = p.v.n_tokens == 0;
    if (!q || !out || (!none && (!kv4_rows(q, &p.q) || !kv4_rows(out, &p.o))) || max_new < 0 || max_len < 0 ||
        window < 0 || !std::isfinite(softmax_scale) || softmax_scale < 0.f || (reinterpret_cast<uintptr_t>(lse) & 3))
        return UW_ERR_INVALID_ARG;
    if (q_heads <= 0 || q_heads % c->kv_heads)
        return UW_ERR_SHAPE;
    if (q_heads > kKv4MaxHeads)
        return UW_ERR_UNSUPPORTED;
    if (none)
        return UW_OK;
    p.lse = lse;
    p.scale = softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt(float(c->head_dim));
    p.q_heads = q_heads;
    p.group = q_heads / c->kv_heads;
    p.causal = causal != 0;
    p.window = window;
    const int64_t blocks = (n_tokens * q_heads + 7) / 8;
    if (blocks > 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (c->head_dim == 128 ? launch_overlapped(kv4_attn_kernel<128>, grid, dim3(256), 0, st, p)
                               : launch_overlapped(kv4_attn_kernel<64>, grid, dim3(256), 0, st, p)) == cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}
