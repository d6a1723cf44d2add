// The 4-bit paged cache of keys and values as the kernels see it: addresses,
// the sequences of a call, and the bounds checks of everything that comes
// from device memory (page numbers, lengths, starts).  The layout is
// described at uw_kv4_cache in include/uw.h.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "decode.cuh"
#include "uw.h"

namespace uw {

// The status word's bit (beside StatusFlag's) for a page number, length or start
// that does not fit the cache or the call.
constexpr uint32_t kStatusBadCache = 16u;

struct Kv4View {
    uint8_t *pages;
    const int32_t *table;
    int64_t n_pages, table_stride;
    const int32_t *start, *len;  // the call's sequences
    int64_t n_tokens;
    int32_t width, n_seqs, heads;
    int32_t page_log2;           // 4 .. 8
    uint32_t *status;
};

struct Rows {
    uint16_t *p;
    int64_t ts, hs;  // token and head strides, in elements
};

// One sequence of a call: its new tokens [t0, t0 + n) and the cached length.
struct Seq {
    int32_t t0, n, len;
};

// Sequence s, with starts outside the call's tokens and lengths beyond the
// table taken as "nothing there" (and reported).
__device__ __forceinline__ Seq kv4_seq(const Kv4View &v, int s) {
    const int32_t a = __ldg(v.start + s), b = __ldg(v.start + s + 1), len = __ldg(v.len + s);
    if (a < 0 || b < a || b > v.n_tokens || len < 0 || int64_t(len) > (int64_t(v.width) << v.page_log2)) {
        atomicOr(v.status, kStatusBadCache);
        return {0, 0, 0};
    }
    return {a, b - a, len};
}

// The (page, kv head) block that holds position p of sequence s; null (and
// reported) for a page outside the pool.
template <int D>
__device__ __forceinline__ uint8_t *kv4_block(const Kv4View &v, int s, int32_t p, int head) {
    const int32_t page = __ldg(v.table + int64_t(s) * v.table_stride + (p >> v.page_log2));
    if (uint32_t(page) >= uint64_t(v.n_pages)) {
        atomicOr(v.status, kStatusBadCache);
        return nullptr;
    }
    return v.pages + (int64_t(page) * v.heads + head) * (int64_t(D + 8) << v.page_log2);
}

// Offsets inside a block of page_size = 1 << pl tokens.
template <int D>
__device__ __forceinline__ uint32_t kv4_codes(int pl, int slot, int is_v) {
    return (uint32_t(is_v) << pl) * (D / 2) + uint32_t(slot) * (D / 2);
}
template <int D>
__device__ __forceinline__ uint32_t kv4_params(int pl, int slot, int is_v) {
    return (uint32_t(D) << pl) + (uint32_t(is_v) << pl) * 4u + uint32_t(slot) * 4u;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Two values rounded to BF16 (nearest even), a in the low half.
__device__ __forceinline__ uint32_t bf16_pack(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Two fp32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Last sequence whose start is at most t, found by the whole warp (every lane
// passes the same t): each round probes 32 evenly spaced starts.
__device__ __forceinline__ int kv4_find_seq(const Kv4View &v, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, span = v.n_seqs;
    while (span > 1) {
        const int step = (span + 31) >> 5;
        const int i = lane * step;
        const bool at_or_before = i < span && __ldg(v.start + lo + i) <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, at_or_before));
        const int skip = c > 0 ? (c - 1) * step : 0;
        lo += skip;
        span = min(step, span - skip);
    }
    return lo;
}

}  // namespace uw
