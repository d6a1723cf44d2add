// Residual addition and root-mean-square norm:
//     h = bf16(x + r),  y = h * (mean(h^2) + eps)^(-1/2) * w
// with y in BF16, or in e4m3 with a scale for each row (largest |y| over 448).
//
// Memory bound: a row is read once, kept in registers as fp32 through the
// sum of squares, and written once.  Rows on 16-byte boundaries with a
// multiple of 8 values up to kMaxVecDim run on 16-byte loads: one warp a row
// up to 1024 values (no barrier; 8 rows a CTA), one CTA a row above.  Rows of
// other sizes, strides or alignments are read value by value, and longer ones
// read again in place of being kept.
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
        const float own = top * rstd / kE4m3Max;
        scale = max_nan(own, kMinScale);
        const bool least = own <= kMinScale, small = top < 1e-30f;  // 448 / top beyond fp32
        a = least ? rstd : small ? 1.f / top : kE4m3Max / top;
        b = least ? 1.f / kMinScale : small ? kE4m3Max : 1.f;
        if (!(own <= INFINITY))
            a = scale;
    }
    __device__ __forceinline__ float of(float u) const { return u * a * b; }
};

// Eight values of h in fp32: x, or with a residual x + r rounded to BF16 and
// stored.
__device__ __forceinline__ void add8(const NormParams &p, int64_t row, int64_t i, const uint4 &xv, const uint4 &rv,
                                     float (&f)[8]) {
    uint32_t a[4] = {xv.x, xv.y, xv.z, xv.w};
    if (p.r) {
        const uint32_t b[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
        for (int k = 0; k < 4; k++)
            a[k] = bf16_pack(bf16_lo(a[k]) + bf16_lo(b[k]), bf16_hi(a[k]) + bf16_hi(b[k]));
        if (p.h && i < p.d)
            *reinterpret_cast<uint4 *>(p.h + row * p.hs + i) = make_uint4(a[0], a[1], a[2], a[3]);
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
        f[2 * k] = bf16_lo(a[k]);
        f[2 * k + 1] = bf16_hi(a[k]);
    }
}

// A row kept in registers by T threads (a warp or a CTA), V vectors of 8 each.
template <int V, bool k8, bool kWarp>
__device__ __forceinline__ void norm_row(const NormParams &p, int64_t row, int t, int T, float *slots) {
    float f[V][8];
    float ss = 0.f;
    // all loads before the first store, which could otherwise not pass it
    uint4 xv[V], w[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int64_t i = 8 * (int64_t(v) * T + t);
        xv[v] = i < p.d ? *reinterpret_cast<const uint4 *>(p.x + row * p.xs + i) : make_uint4(0, 0, 0, 0);
        w[v] = i < p.d && p.r ? *reinterpret_cast<const uint4 *>(p.r + row * p.rs + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int64_t i = 8 * (int64_t(v) * T + t);
        add8(p, row, i, xv[v], w[v], f[v]);
#pragma unroll
        for (int k = 0; k < 8; k++)
            ss = fmaf(f[v][k], f[v][k], ss);
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int64_t i = 8 * (int64_t(v) * T + t);
        w[v] = i < p.d ? __ldg(reinterpret_cast<const uint4 *>(p.w + i)) : make_uint4(0, 0, 0, 0);
    }
    ss = kWarp ? warp_sum(ss) : cta_reduce<false>(ss, slots);
    const float rstd = rsqrtf(ss / float(p.d) + p.eps);
    float top = 0.f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int64_t i = 8 * (int64_t(v) * T + t);
        const uint32_t wv[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
        if (i < p.d) {
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
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + row * p.ys + i) =
                    make_uint4(bf16_pack(f[v][0] * rstd, f[v][1] * rstd), bf16_pack(f[v][2] * rstd, f[v][3] * rstd),
                               bf16_pack(f[v][4] * rstd, f[v][5] * rstd), bf16_pack(f[v][6] * rstd, f[v][7] * rstd));
            }
        }
    }
    if constexpr (k8) {
        const RowScale s(kWarp ? warp_max(top) : cta_reduce<true>(top, slots + 32), rstd);
        if (t == 0)
            p.scale[row] = s.scale;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int64_t i = 8 * (int64_t(v) * T + t);
            if (i < p.d) {
                uint32_t q[2];
#pragma unroll
                for (int k = 0; k < 2; k++)
                    q[k] = to_e4m3x2(s.of(f[v][4 * k]), s.of(f[v][4 * k + 1])) |
                           uint32_t(to_e4m3x2(s.of(f[v][4 * k + 2]), s.of(f[v][4 * k + 3]))) << 16;
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.y) + row * p.ys + i) = make_uint2(q[0], q[1]);
            }
        }
    }
}

template <int V, bool k8>
__global__ void __launch_bounds__(256) norm_warp_kernel(const NormParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row < p.n)
        norm_row<V, k8, true>(p, row, threadIdx.x & 31, 32, nullptr);
}

template <int V, bool k8>
__global__ void __launch_bounds__(512) norm_cta_kernel(const NormParams p) {
    __shared__ float slots[64];
    grid_dep_launch();
    grid_dep_wait();
    norm_row<V, k8, false>(p, blockIdx.x, threadIdx.x, blockDim.x, slots);
}

// Rows whose size, stride or alignment is not one of 16-byte loads, up to V
// values a thread: the same with single values, thread t of T having t, t + T, ...
template <int V, bool k8>
__global__ void __launch_bounds__(512) norm_odd_kernel(const NormParams p) {
    __shared__ float slots[64];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t row = blockIdx.x;
    const int d = int(p.d), T = blockDim.x;
    const uint16_t *x = p.x + row * p.xs, *r = p.r ? p.r + row * p.rs : nullptr;
    uint16_t *h = p.h ? p.h + row * p.hs : nullptr;
    // all loads before the first store, which could otherwise not pass it
    float f[V], w[V], ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int i = v * T + int(threadIdx.x);
        f[v] = i < d ? bf16_lo(x[i]) : 0.f;
    }
    if (r) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int i = v * T + int(threadIdx.x);
            w[v] = i < d ? bf16_lo(r[i]) : 0.f;
        }
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int i = v * T + int(threadIdx.x);
            const __nv_bfloat16 b = __float2bfloat16_rn(f[v] + w[v]);
            if (h && i < d)
                h[i] = __bfloat16_as_ushort(b);
            f[v] = __bfloat162float(b);
        }
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int i = v * T + int(threadIdx.x);
        w[v] = i < d ? bf16_lo(p.w[i]) : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; v++)
        ss = fmaf(f[v], f[v], ss);
    const float rstd = rsqrtf(cta_reduce<false>(ss, slots) / float(d) + p.eps);
    float top = 0.f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int i = v * T + int(threadIdx.x);
        if (i < d) {
            f[v] *= w[v];
            if constexpr (k8)
                top = max_nan(top, fabsf(f[v]));
            else
                static_cast<uint16_t *>(p.y)[row * p.ys + i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[v] * rstd));
        }
    }
    if constexpr (k8) {
        const RowScale s(cta_reduce<true>(top, slots + 32), rstd);
        if (threadIdx.x == 0)
            p.scale[row] = s.scale;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int i = v * T + int(threadIdx.x);
            if (i < d)
                static_cast<uint8_t *>(p.y)[row * p.ys + i] = to_e4m3(s.of(f[v]));
        }
    }
}

// Longer rows of any kind: the row is walked value by value, and x and r read
// again for the second and third pass.
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

template <bool k8>
cudaError_t launch_norm(const NormParams &p, bool vec, cudaStream_t st) {
    if (!vec && p.d <= kMaxVecDim) {
        const int v = p.d <= 8 * 512 ? 8 : p.d <= 16 * 512 ? 16 : 32;
        const dim3 grid(unsigned(p.n)), block(unsigned((p.d + 32 * v - 1) / (32 * v) * 32));
        return v == 8    ? launch_overlapped(norm_odd_kernel<8, k8>, grid, block, 0, st, p)
               : v == 16 ? launch_overlapped(norm_odd_kernel<16, k8>, grid, block, 0, st, p)
                         : launch_overlapped(norm_odd_kernel<32, k8>, grid, block, 0, st, p);
    }
    if (p.d > kMaxVecDim)
        return launch_overlapped(norm_any_kernel<k8>, dim3(unsigned(p.n)), dim3(512), 0, st, p);
    const int vecs = int(p.d / 8);
    if (p.d <= kWarpDim) {
        const dim3 grid(unsigned((p.n + 7) / 8)), block(256);
        if (vecs <= 32)
            return launch_overlapped(norm_warp_kernel<1, k8>, grid, block, 0, st, p);
        if (vecs <= 64)
            return launch_overlapped(norm_warp_kernel<2, k8>, grid, block, 0, st, p);
        return launch_overlapped(norm_warp_kernel<4, k8>, grid, block, 0, st, p);
    }
    const dim3 grid(static_cast<unsigned>(p.n));
    if (vecs <= 512)
        return launch_overlapped(norm_cta_kernel<2, k8>, grid, dim3((vecs + 63) / 64 * 32), 0, st, p);
    if (vecs <= 1024)
        return launch_overlapped(norm_cta_kernel<4, k8>, grid, dim3((vecs + 127) / 128 * 32), 0, st, p);
    return launch_overlapped(norm_cta_kernel<8, k8>, grid, dim3((vecs + 255) / 256 * 32), 0, st, p);
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
    bool vec = d % 8 == 0 && (bits16 & 15) == 0 && (reinterpret_cast<uintptr_t>(y) & (k8 ? 7 : 15)) == 0;
    if (n > 1)
        vec = vec && xs % 8 == 0 && ys % 8 == 0 && (!r || rs % 8 == 0) && (!h || hs % 8 == 0);
    const NormParams p{x, r, w, h, y, scale, xs, rs, hs, ys, n, d, eps};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (k8 ? launch_norm<true>(p, vec, st) : launch_norm<false>(p, vec, st)) == cudaSuccess ? UW_OK : UW_ERR_CUDA;
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
