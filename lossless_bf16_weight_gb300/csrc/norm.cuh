// What the norm kernels share: sums and maxima over a warp or a CTA, the 8-bit
// form of a row, and 16-byte steps over rows that may begin anywhere.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "kv4.cuh"

namespace uw {

constexpr int kWarpDim = 1024;     // longest row of one warp: 4 vectors of 8 a lane
constexpr int kMaxVecDim = 16384;  // longest row kept in registers
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

// max that keeps NaN, so that a row's NaN reaches its scale
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Sum (or maximum) over the CTA; every thread gets it.  `slot`: 32 floats not
// in use by an earlier call that some thread may still read.
template <bool kMax>
__device__ __forceinline__ float cta_reduce(float v, float *slot) {
    const int nw = (blockDim.x + 31) >> 5;
    v = kMax ? warp_max(v) : warp_sum(v);
    if ((threadIdx.x & 31) == 0)
        slot[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = int(threadIdx.x & 31) < nw ? slot[threadIdx.x & 31] : 0.f;
    return kMax ? warp_max(t) : warp_sum(t);
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
    return uint8_t(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint16_t to_e4m3x2(float a, float b) {
    return uint16_t(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// The 8-bit form of a row from u = h * w (exact in fp32: 8 x 8 significant
// bits; with an offset of the weights the sum and the product are rounded) and its largest magnitude.  1 / rms stands in y
// and in the scale and cancels in y / scale = u * (448 / max |u|), so a code depends on no sum over the row and on
// two roundings beside those of u.  A row whose scale is the smallest (max |y| below 448 *
// 2^-126) takes y times 2^126; one that is not finite, or whose u is not, has a
// NaN scale.
struct RowScale {
    float scale, a, b;
    __device__ __forceinline__ RowScale(float top, float rstd) {
        float own = top * rstd / kE4m3Max;
        own = own < INFINITY ? own : __int_as_float(0x7fffffff);  // NaN stays NaN
        scale = max_nan(own, kMinScale);
        const bool least = own <= kMinScale, small = top < 1e-30f;  // 448 / top beyond fp32
        a = least ? rstd : small ? 1.f / top : kE4m3Max / top;
        b = least ? 1.f / kMinScale : small ? kE4m3Max : 1.f;
        if (!(own < INFINITY))
            a = scale;
    }
    __device__ __forceinline__ float of(float u) const { return u * a * b; }
};

// Eight values from i on of row `row` of n rows of d values, one access.  kOdd: a row's first
// and last eight may be only partly its own (i may be below 0): the others are its
// neighbours', or between the rows, and left out.
template <bool kOdd>
__device__ __forceinline__ uint4 load8(const uint16_t *all, int64_t stride, int64_t n, int64_t d, int64_t row,
                                       int64_t i) {
    const uint16_t *const at = all + (row * stride + i);
    if (i >= d || (kOdd && i + 8 <= 0))
        return make_uint4(0, 0, 0, 0);
    if (!kOdd || (i >= 0 && i + 8 <= d))
        return *reinterpret_cast<const uint4 *>(at);
    uint32_t a[4] = {0, 0, 0, 0};
    const int lo = i < 0 ? int(-i) : 0, hi = d - i < 8 ? int(d - i) : 8;
    if (row * stride + i >= 0 && row * stride + i + 8 <= (n - 1) * stride + d) {
        const uint4 x = *reinterpret_cast<const uint4 *>(at);
        a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
#pragma unroll
        for (int k = 0; k < 4; k++)
            a[k] &= (2 * k >= lo && 2 * k < hi ? 0xffffu : 0u) | (2 * k + 1 >= lo && 2 * k + 1 < hi ? 0xffff0000u : 0u);
    } else {
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (k >= lo && k < hi)
                a[k / 2] |= uint32_t(at[k]) << (16 * (k & 1));
    }
    return make_uint4(a[0], a[1], a[2], a[3]);
}
template <bool kOdd>
__device__ __forceinline__ void store8(uint16_t *row, int64_t i, int64_t d, const uint32_t (&a)[4]) {
    if (kOdd ? i >= 0 && i + 8 <= d : i < d) {
        *reinterpret_cast<uint4 *>(row + i) = make_uint4(a[0], a[1], a[2], a[3]);
    } else if (kOdd && i + 8 > 0 && i < d) {
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (i + k >= 0 && i + k < d)
                row[i + k] = uint16_t(a[k / 2] >> (16 * (k & 1)));
    }
}
template <bool kOdd>
__device__ __forceinline__ void store8(uint8_t *row, int64_t i, int64_t d, const uint32_t (&a)[2]) {
    if (kOdd ? i >= 0 && i + 8 <= d : i < d) {
        *reinterpret_cast<uint2 *>(row + i) = make_uint2(a[0], a[1]);
    } else if (kOdd && i + 8 > 0 && i < d) {
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (i + k >= 0 && i + k < d)
                row[i + k] = uint8_t(a[k / 4] >> (8 * (k & 3)));
    }
}
// The same of the weights, which begin at a distance of their own from a
// 16-byte step: two steps, shifted into place, or in short rows (a warp's), whose
// ends cannot be, value by value (30000 x 257 25 us, shifted 29; 8000 x 1001 13.3 and 13.7).
template <bool kOdd, bool kWarp>
__device__ __forceinline__ uint4 load8_weights(const uint16_t *w, int64_t i, int64_t d) {
    if constexpr (!kOdd) {
        return i < d ? __ldg(reinterpret_cast<const uint4 *>(w + i)) : make_uint4(0, 0, 0, 0);
    } else {
        const int off = int(uint32_t(i) + uint32_t(reinterpret_cast<uintptr_t>(w) >> 1)) & 7;
        const int64_t from = i - off;
        if (!kWarp && from >= 0 && from + 16 <= d) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(w + from));
            const uint4 y = __ldg(reinterpret_cast<const uint4 *>(w + from) + 1);
            uint32_t a[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 6; k++)
                a[k] = off & 4 ? a[k + 2] : a[k];
#pragma unroll
            for (int k = 0; k < 5; k++)
                a[k] = off & 2 ? a[k + 1] : a[k];
            const uint32_t sel = off & 1 ? 0x5432u : 0x3210u;
            return make_uint4(__byte_perm(a[0], a[1], sel), __byte_perm(a[1], a[2], sel), __byte_perm(a[2], a[3], sel),
                              __byte_perm(a[3], a[4], sel));
        }
        uint32_t a[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (i + k >= 0 && i + k < d)
                a[k / 2] |= uint32_t(__ldg(w + i + k)) << (16 * (k & 1));
        return make_uint4(a[0], a[1], a[2], a[3]);
    }
}

}  // namespace uw
