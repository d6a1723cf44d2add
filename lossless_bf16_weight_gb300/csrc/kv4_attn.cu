// Entry points of the 4-bit paged cache's attention, and the checks of what the
// cache's calls are given.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kernels.h"
#include "kv4_attn.cuh"
#include "kv4_codes.cuh"
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

// Sequences with up to so many rows (new tokens x query heads of a kv head)
// take the kernel for few rows: kFewRows, or what a call of kShort units (32 keys
// x 8 rows) in all makes, up to kFewRowsShort (whose row tiles a CTA looks through
// one by one).  That kernel and the other, 8 kv heads of 128: 16 sequences of 4096 keys, 16
// rows 41 and 82 us, 32 rows 65 and 81, 64 rows 110 and 83; one sequence of 8192 keys, 64
// rows 29 and 48; of 1000 keys, 256 rows 23 and 32, 512 rows 32 and 34, 1024 rows 44 and 35;
// prompts of 64 tokens of 4 heads 10.9 and 17.2, of 128 17.0 and 17.9, of 512 43 and 29.
constexpr int kFewRows = 32, kFewRowsShort = 1024;
constexpr int64_t kShort = 24576;

// Workspace: [error word | counters of the kernel for few rows | of the other |
// parts of the one | of the other].  The counters, which a call finds at zero, lie in
// the same place for every head size, so that one workspace serves both.
struct Layout {
    size_t few_counters, many_counters, few_parts, many_parts, total;
};
Layout layout(int head_dim) {
    Layout w;
    w.few_counters = 256;
    w.many_counters = align_up(w.few_counters + 4 * size_t(kv4_decode_ctas()), 256);
    w.few_parts = align_up(w.many_counters + 4 * size_t(kv4_prefill_ctas()), 256);
    w.many_parts = align_up(w.few_parts + 4 * kv4_decode_part_floats(head_dim), 256);
    w.total = w.many_parts + 4 * kv4_prefill_part_floats(head_dim);
    return w;
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
    if (c->head_dim != 64 && c->head_dim != 128)
        return UW_ERR_UNSUPPORTED;
    *bytes = layout(c->head_dim).total;
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
    p.c1 = (softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt(float(c->head_dim))) * 1.44269504089f;
    if (q_heads > kKv4MaxHeads || n_tokens * (q_heads / c->kv_heads) > 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    // the kernels take codes in units of 2^-133 and so multiply by c1 * kQDown
    if (!(p.c1 >= FLT_MIN) || !std::isfinite(p.c1 * kQDown))
        return UW_ERR_UNSUPPORTED;
    if (none)
        return UW_OK;
    const Layout w = layout(c->head_dim);
    if (ws_bytes < w.total)
        return UW_ERR_BUFFER_TOO_SMALL;
    p.lse = lse;
    p.q_heads = q_heads;
    p.group = q_heads / c->kv_heads;
    p.by_group = Divisor(uint32_t(p.group));
    p.out32 = ((reinterpret_cast<uintptr_t>(p.o.p) | uintptr_t(p.o.ts) * 2 | uintptr_t(p.o.hs) * 2) & 31) == 0;
    p.causal = causal != 0;
    p.window = window;
    uint8_t *const wsb = static_cast<uint8_t *>(ws);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Which sequences take which kernel is decided on the device by their rows;
    // the host's bounds only leave out a launch that has none, and a wrong bound
    // leaves all sequences to the kernel that is launched.
    const int64_t rows = std::min<int64_t>(max_new, INT32_MAX) * p.group;
    // units of eight rows of each sequence (bounds may be any number)
    const int64_t of_one = (std::min<int64_t>(max_len, INT32_MAX) / 32 + 2) * c->kv_heads;
    const int64_t eight = std::min<int64_t>(std::min<int64_t>(of_one, INT32_MAX) * c->n_seqs, 1ll << 40);
    const int few_rows = max_len > 0 ? int(std::clamp<int64_t>(kShort / eight * 8, kFewRows, kFewRowsShort)) : kFewRows;
    const bool few = rows == 0 || rows <= few_rows || c->n_seqs > 1, many = rows == 0 || rows > few_rows;
    if (few) {
        p.rows_min = 0;
        p.rows_max = many ? few_rows : INT32_MAX;
        p.counters = reinterpret_cast<uint32_t *>(wsb + w.few_counters);
        p.parts = reinterpret_cast<float *>(wsb + w.few_parts);
        const int64_t units = max_len > 0 && !many ? eight * (rows / 8 + 1) : 0;
        // beside prompts most of the other sequences have one new token
        const uw_status r = launch_kv4_decode(p, c->head_dim, many ? std::max(p.group, 5) : rows, units, st);
        if (r != UW_OK)
            return r;
    }
    if (many) {
        p.rows_min = few ? few_rows + 1 : 0;
        p.rows_max = INT32_MAX;
        p.counters = reinterpret_cast<uint32_t *>(wsb + w.many_counters);
        p.parts = reinterpret_cast<float *>(wsb + w.many_parts);
        return launch_kv4_prefill(p, c->head_dim, st);
    }
    return UW_OK;
}
