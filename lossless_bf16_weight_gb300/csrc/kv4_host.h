// Host-side checks and workspace layout shared by the entry points of the
// 4-bit paged cache.
#pragma once
#include <cstddef>
#include <cstdint>

#include "kv4.cuh"

namespace uw {

constexpr int kKv4MaxHeads = 1 << 16;

// What a call passes, checked, as the kernels take it.
uw_status kv4_view(const uw_kv4_cache *c, const int32_t *start, const int32_t *len, int64_t n_tokens, void *ws,
                   size_t ws_bytes, Kv4View *v);
// 16-byte aligned rows with strides of whole 16-byte steps.
bool kv4_rows(const uw_kv4_rows *r, Rows *out);

}  // namespace uw
