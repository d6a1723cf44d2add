// Residual addition and root-mean-square norm:
//     h = bf16(x + r),  y = h * (mean(h^2) + eps)^(-1/2) * w
// with y in BF16, or in e4m3 with a scale for each row (largest |y| over 448).
//
// Memory bound: a row is read once, kept in registers as fp32 through the
// sum of squares, and written once, in 16-byte steps: one warp a row up to
// 1024 values (no barrier; 8 rows a CTA), one CTA a row above.  Rows may begin
// anywhere, if x, r, h and y do so alike (tensors of odd rows do): their vectors
// lie on the steps around a row, and what is not the row's is left out.  Rows
// that do not, and those of more than 16384 values, are taken value by value
// and read again for each pass.
//
// Measured, with a residual, to BF16 unless stated:
//   1 x 4096               1.5 us
//   257 x 4096 to 8 bits   3.1 us (2.3 TB/s)
//   8192 x 4096            40 us (6.7 TB/s, of 6.8 for a copy)
//   8192 x 4097            52 us (5.2 TB/s); value by value 80
//   8192 x 1024            9.8 us (in L2); by a CTA a row 10.0, 30000 x 256 8.1 and 30.8
//   2000 x 16384 to 8 bits 38 us (6.1 TB/s); value by value 94
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "kv4.cuh"

namespace uw {

namespace {

constexpr int kWarpDim = 1024;     // longest row of one warp: 4 vectors of 8 a lane
constexpr int kMaxVecDim = 16384;  // longest row kept in registers: 256 threads x 8 vectors of 8
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

struct NormParams {
    const uint16_t *x, *r, *w;
    uint16_t *h;
    void *y;
    float *scale;
    int64_t xs, rs, hs, ys, n, d;
    float eps;
};

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
// bits) and its largest magnitude.  1 / rms stands in y and in the scale and
// cancels in y / scale = u * (448 / max |u|), so a code depends on two
// roundings only.  A row whose scale is the smallest (max |y| below 448 *
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

// Eight values from i on of a row of d values, one access.  kOdd: a row's first
// and last eight may be only partly its own (i may be below 0): the others are its
// neighbours', or between the rows, and left out.
template <bool kOdd>
__device__ __forceinline__ uint4 load8(const uint16_t *all, int64_t stride, const NormParams &p, int64_t row,
                                       int64_t i) {
    const int64_t d = p.d;
    const uint16_t *const at = all + (row * stride + i);
    if (i >= d || (kOdd && i + 8 <= 0))
        return make_uint4(0, 0, 0, 0);
    if (!kOdd || (i >= 0 && i + 8 <= d))
        return *reinterpret_cast<const uint4 *>(at);
    uint32_t a[4] = {0, 0, 0, 0};
    const int lo = i < 0 ? int(-i) : 0, hi = d - i < 8 ? int(d - i) : 8;
    if (row * stride + i >= 0 && row * stride + i + 8 <= (p.n - 1) * stride + d) {
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

// Eight values of h in fp32: x, or with a residual x + r rounded to BF16 and
// stored.
template <bool kOdd>
__device__ __forceinline__ void add8(const NormParams &p, int64_t row, int64_t i, const uint4 &xv, const uint4 &rv,
                                     float (&f)[8]) {
    uint32_t a[4] = {xv.x, xv.y, xv.z, xv.w};
    if (p.r) {
        const uint32_t b[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
        for (int k = 0; k < 4; k++)
            a[k] = bf16_pack(bf16_lo(a[k]) + bf16_lo(b[k]), bf16_hi(a[k]) + bf16_hi(b[k]));
        if (p.h)
            store8<kOdd>(p.h + row * p.hs, i, p.d, a);
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
        f[2 * k] = bf16_lo(a[k]);
        f[2 * k + 1] = bf16_hi(a[k]);
    }
}

// A row kept in registers by T threads (a warp or a CTA), V vectors of 8 each.
// kOdd: the row begins anywhere; its vectors lie on the 16-byte steps around
// it (of x, and at the same distance of r, h and y).
template <int V, bool k8, bool kWarp, bool kOdd>
__device__ __forceinline__ void norm_row(const NormParams &p, int64_t row, int t, int T, float *slots) {
    const int before = kOdd ? int(reinterpret_cast<uintptr_t>(p.x + row * p.xs) >> 1) & 7 : 0;
    auto first = [&](int v) { return 8 * (int64_t(v) * T + t) - before; };
    float f[V][8];
    float ss = 0.f;
    // all loads before the first store, which could otherwise not pass it
    uint4 xv[V], w[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        xv[v] = load8<kOdd>(p.x, p.xs, p, row, first(v));
        w[v] = p.r ? load8<kOdd>(p.r, p.rs, p, row, first(v)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
        add8<kOdd>(p, row, first(v), xv[v], w[v], f[v]);
#pragma unroll
        for (int k = 0; k < 8; k++)
            ss = fmaf(f[v][k], f[v][k], ss);
    }
    if constexpr (!kOdd) {  // (value by value they would take the registers of a long row)
#pragma unroll
        for (int v = 0; v < V; v++)
            w[v] = load8_weights<kOdd, kWarp>(p.w, first(v), p.d);
    }
    ss = kWarp ? warp_sum(ss) : cta_reduce<false>(ss, slots);
    const float rstd = rsqrtf(ss / float(p.d) + p.eps);
    float top = 0.f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        if constexpr (kOdd)
            w[v] = load8_weights<kOdd, kWarp>(p.w, first(v), p.d);
        const uint32_t wv[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            f[v][2 * k] *= bf16_lo(wv[k]);
            f[v][2 * k + 1] *= bf16_hi(wv[k]);
        }
        if constexpr (k8) {
#pragma unroll
            for (int k = 0; k < 8; k++)
                top = max_nan(top, fabsf(f[v][k]));
        } else {
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; k++)
                y[k] = bf16_pack(f[v][2 * k] * rstd, f[v][2 * k + 1] * rstd);
            store8<kOdd>(static_cast<uint16_t *>(p.y) + row * p.ys, first(v), p.d, y);
        }
    }
    if constexpr (k8) {
        const RowScale s(kWarp ? warp_max(top) : cta_reduce<true>(top, slots + 32), rstd);
        if (t == 0)
            p.scale[row] = s.scale;
#pragma unroll
        for (int v = 0; v < V; v++) {
            uint32_t q[2];
#pragma unroll
            for (int k = 0; k < 2; k++)
                q[k] = to_e4m3x2(s.of(f[v][4 * k]), s.of(f[v][4 * k + 1])) |
                       uint32_t(to_e4m3x2(s.of(f[v][4 * k + 2]), s.of(f[v][4 * k + 3]))) << 16;
            store8<kOdd>(static_cast<uint8_t *>(p.y) + row * p.ys, first(v), p.d, q);
        }
    }
}

template <int V, bool k8, bool kOdd>
__global__ void __launch_bounds__(256) norm_warp_kernel(const NormParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row < p.n)
        norm_row<V, k8, true, kOdd>(p, row, threadIdx.x & 31, 32, nullptr);
}

// (Rows of up to 16384 that begin anywhere take up to 288 threads, two CTAs an SM: 2000
// x 16383 to 8 bits 65 us, one CTA 103.)
template <int V, bool k8, bool kOdd>
__global__ void __launch_bounds__(kOdd && V == 8 ? 288 : 512, kOdd && V == 8 ? 2 : 0)
    norm_cta_kernel(const NormParams p) {
    __shared__ float slots[64];
    grid_dep_launch();
    grid_dep_wait();
    norm_row<V, k8, false, kOdd>(p, blockIdx.x, threadIdx.x, blockDim.x, slots);
}

// Rows of any kind, value by value, with x and r read again for the second and
// third pass.
template <bool k8>
__global__ void __launch_bounds__(512) norm_any_kernel(const NormParams p) {
    __shared__ float slots[64];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t row = blockIdx.x;
    const uint16_t *x = p.x + row * p.xs, *r = p.r ? p.r + row * p.rs : nullptr;
    uint16_t *h = p.h ? p.h + row * p.hs : nullptr;
    auto value = [&](int64_t i) {
        float f = bf16_lo(x[i]);
        if (r)
            f = __bfloat162float(__float2bfloat16_rn(f + bf16_lo(r[i])));
        return f;
    };
    float ss = 0.f;
    for (int64_t i = threadIdx.x; i < p.d; i += blockDim.x) {
        const float f = value(i);
        ss = fmaf(f, f, ss);
    }
    const float rstd = rsqrtf(cta_reduce<false>(ss, slots) / float(p.d) + p.eps);
    float top = 0.f;
    if constexpr (k8) {
        for (int64_t i = threadIdx.x; i < p.d; i += blockDim.x)
            top = max_nan(top, fabsf(value(i) * bf16_lo(p.w[i])));
        top = cta_reduce<true>(top, slots + 32);
    }
    const RowScale s(top, rstd);
    if (k8 && threadIdx.x == 0)
        p.scale[row] = s.scale;
    for (int64_t i = threadIdx.x; i < p.d; i += blockDim.x) {
        const float f = value(i), u = f * bf16_lo(p.w[i]);
        if (h && r)
            h[i] = __bfloat16_as_ushort(__float2bfloat16_rn(f));  // after the last read of x[i] and r[i]
        if constexpr (k8)
            static_cast<uint8_t *>(p.y)[row * p.ys + i] = to_e4m3(s.of(u));
        else
            static_cast<uint16_t *>(p.y)[row * p.ys + i] = __bfloat16_as_ushort(__float2bfloat16_rn(u * rstd));
    }
}

template <bool k8, bool kOdd>
cudaError_t launch_rows(const NormParams &p, cudaStream_t st) {
    const int vecs = int((p.d + (kOdd ? 14 : 7)) / 8);  // vectors of a row, wherever it begins
    if (vecs <= kWarpDim / 8) {
        const dim3 grid(unsigned((p.n + 7) / 8)), block(256);
        if (vecs <= 32)
            return launch_overlapped(norm_warp_kernel<1, k8, kOdd>, grid, block, 0, st, p);
        if (vecs <= 64)
            return launch_overlapped(norm_warp_kernel<2, k8, kOdd>, grid, block, 0, st, p);
        return launch_overlapped(norm_warp_kernel<4, k8, kOdd>, grid, block, 0, st, p);
    }
    const dim3 grid(static_cast<unsigned>(p.n));
    if (vecs <= 512)
        return launch_overlapped(norm_cta_kernel<2, k8, kOdd>, grid, dim3((vecs + 63) / 64 * 32), 0, st, p);
    if (vecs <= 1024)
        return launch_overlapped(norm_cta_kernel<4, k8, kOdd>, grid, dim3((vecs + 127) / 128 * 32), 0, st, p);
    return launch_overlapped(norm_cta_kernel<8, k8, kOdd>, grid, dim3((vecs + 255) / 256 * 32), 0, st, p);
}

// vec: every row begins on a step of eight values; alike: the rows of x, r, h and y
// begin at the same distance from one.
template <bool k8>
cudaError_t launch_norm(const NormParams &p, bool vec, bool alike, cudaStream_t st) {
    if (p.d > kMaxVecDim || !alike)
        return launch_overlapped(norm_any_kernel<k8>, dim3(unsigned(p.n)), dim3(512), 0, st, p);
    return vec ? launch_rows<k8, false>(p, st) : launch_rows<k8, true>(p, st);
}

uw_status run_norm(const uint16_t *x, int64_t xs, const uint16_t *r, int64_t rs, uint16_t *h, int64_t hs,
                   const uint16_t *w, int64_t n, int64_t d, float eps, void *y, int64_t ys, float *scale, bool k8,
                   void *stream) {
    // no rows need no buffers (those of empty tensors are null)
    if ((n != 0 && (!x || !w || !y || (k8 && !scale))) || n < 0 || (h && !r) || !(eps >= 0.f))
        return UW_ERR_INVALID_ARG;
    if (d <= 0)
        return UW_ERR_SHAPE;
    if (n > 0x7fffffff || d > 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    if (n > 1 && (xs < d || ys < d || (r && rs < d) || (h && hs < d)))
        return UW_ERR_INVALID_ARG;
    if (n == 0)
        return UW_OK;
    const uintptr_t bits16 = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(r) |
                             reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(w);
    if ((bits16 & 1) || (!k8 && (reinterpret_cast<uintptr_t>(y) & 1)) ||
        (k8 && (reinterpret_cast<uintptr_t>(scale) & 3)))
        return UW_ERR_INVALID_ARG;
    // where a tensor's rows begin, in values: eight of them are 16 bytes (8 of e4m3)
    const uint64_t x0 = reinterpret_cast<uintptr_t>(x) / 2, y0 = reinterpret_cast<uintptr_t>(y) / (k8 ? 1 : 2);
    auto as_x = [&](uint64_t first, int64_t stride) {
        return (first - x0) % 8 == 0 && (n == 1 || (stride - xs) % 8 == 0);
    };
    const bool alike = as_x(y0, ys) && (!r || as_x(reinterpret_cast<uintptr_t>(r) / 2, rs)) &&
                       (!h || as_x(reinterpret_cast<uintptr_t>(h) / 2, hs));
    const bool vec = d % 8 == 0 && x0 % 8 == 0 && (n == 1 || xs % 8 == 0) && reinterpret_cast<uintptr_t>(w) % 16 == 0;
    const NormParams p{x, r, w, h, y, scale, xs, rs, hs, ys, n, d, eps};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (k8 ? launch_norm<true>(p, vec, alike, st) : launch_norm<false>(p, vec, alike, st)) == cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}

}  // namespace
}  // namespace uw

extern "C" uw_status uw_rmsnorm(const uint16_t *x, int64_t xs, const uint16_t *r, int64_t rs, uint16_t *h, int64_t hs,
                                const uint16_t *w, int64_t n, int64_t d, float eps, uint16_t *y, int64_t ys,
                                void *stream) {
    return uw::run_norm(x, xs, r, rs, h, hs, w, n, d, eps, y, ys, nullptr, false, stream);
}

extern "C" uw_status uw_rmsnorm_e4m3(const uint16_t *x, int64_t xs, const uint16_t *r, int64_t rs, uint16_t *h,
                                     int64_t hs, const uint16_t *w, int64_t n, int64_t d, float eps, uint8_t *q,
                                     int64_t qs, float *scale, void *stream) {
    return uw::run_norm(x, xs, r, rs, h, hs, w, n, d, eps, q, qs, scale, true, stream);
}
