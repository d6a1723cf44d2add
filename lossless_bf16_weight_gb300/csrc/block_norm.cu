// The norms around a block of a layer, with its gate, scales and residual sum:
//     z = x, or x (mean(x^2) + eps)^(-1/2) (wp + off)
//     h = bf16(rs r + bs g z)
//     y = h (mean(h^2) + eps)^(-1/2) (w + off)
// with y in BF16, or in e4m3 with a scale for each row, or left out.
//
// Memory bound, and with 35 instructions issued a value not far from bound by issue slots (74% of them): x, r
// (and a gate of every row) are read once, h and y written once, in 16-byte steps; a row stays in
// registers through its two sums, x and r as they came.  One warp a row up to 1024 values, one CTA a row above,
// rows that may begin anywhere as in norm.cu; rows that are not alike or have more than 16384 values are
// taken value by value, with h read back (or made again) for the second norm.
//
// Measured in a graph, with a norm after the block and a gate for all rows unless stated (of 6.8 TB/s for a copy):
//   1 x 4096, no gate      2.2 us
//   257 x 5120 to 8 bits   3.9 us
//   8191 x 4096            42.3 us (6.35 TB/s); to 8 bits 44.9 (5.2); a gate of every row 49.9 (6.7)
//   16000 x 2048           39.7 us (6.6 TB/s)
//   4000 x 8192            43.4 us (6.0 TB/s); 2000 x 16384 45.1 (5.8)
//   8000 x 1000            9.5 us (in L2); 8000 x 1001 21.7
//   8000 x 4097            82.7 us (3.2 TB/s: three weights a value shifted into place)
// One CTA for many rows, weights and gate kept in registers and the next row's x and r on their way: 55 us
// for 8191 x 4096 (its registers leave too few warps).
#include <cmath>

#include "norm.cuh"

namespace uw {

namespace {

struct BlockParams {
    const uint16_t *x, *r, *g, *wp, *w;
    uint16_t *h;
    void *y;
    float *scale;
    int64_t xs, rs, gs, hs, ys, n, d;  // gs 0: one gate for all rows
    float eps, off, r_scale, b_scale;
    float minus_zero;                 // -0, which the compiler does not know
};

// Two values each: a b + c with the products of BF16 pairs exact, and a + c, by the instructions that take BF16 as
// it is (a conversion for each value otherwise, which with three reads and two sums of a value is what issue slots
// go to: 8191 x 4096 3% more without).
__device__ __forceinline__ void fma_pair(uint32_t a, uint32_t b, float &c0, float &c1) {
    asm("{\n\t.reg .b16 al, ah, bl, bh;\n\t"
        "mov.b32 {al, ah}, %2;\n\t"
        "mov.b32 {bl, bh}, %3;\n\t"
        "fma.rn.f32.bf16 %0, al, bl, %0;\n\t"
        "fma.rn.f32.bf16 %1, ah, bh, %1;\n\t}"
        : "+f"(c0), "+f"(c1)
        : "r"(a), "r"(b));
}
__device__ __forceinline__ float2 add_pair(uint32_t a, float c) {
    float2 r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "add.rn.f32.bf16 %0, l, %3;\n\t"
        "add.rn.f32.bf16 %1, h, %3;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(a), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int k) { return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w; }

// A row kept in registers by T threads (a warp or a CTA), V vectors of 8 each.
// kOdd: the row begins anywhere (norm.cuh).  kLate: weights and gate are loaded where they are used.
template <int V, bool k8, bool kWarp, bool kOdd, bool kLate = kOdd>
__device__ __forceinline__ void block_row(const BlockParams &p, int64_t row, int t, int T, float *slots) {
    const int before = kOdd ? int(reinterpret_cast<uintptr_t>(p.x + row * p.xs) >> 1) & 7 : 0;
    auto first = [&](int v) { return 8 * (int64_t(v) * T + t) - before; };
    auto weights = [&](const uint16_t *w, int v) { return load8_weights<kOdd, kWarp>(w, first(v), p.d); };
    auto gates = [&](int v) {
        return p.gs ? load8<kOdd>(p.g, p.gs, p.n, p.d, row, first(v)) : weights(p.g, v);
    };
    // the row's loads before the first store, which could otherwise not pass it
    uint4 x[V], r[V], a[V], g[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        x[v] = load8<kOdd>(p.x, p.xs, p.n, p.d, row, first(v));
        r[v] = load8<kOdd>(p.r, p.rs, p.n, p.d, row, first(v));
    }
    if constexpr (!kLate) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (p.g)
                g[v] = gates(v);
            if (p.wp)
                a[v] = weights(p.wp, v);
        }
    }
    float c = p.b_scale;  // of x
    if (p.wp) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int k = 0; k < 4; k++)
                fma_pair(word(x[v], k), word(x[v], k), s0, s1);
        const float ss = kWarp ? warp_sum(s0 + s1) : cta_reduce<false>(s0 + s1, slots);
        c *= rsqrtf(ss / float(p.d) + p.eps);
    }
    const uint64_t zero = pair2(p.minus_zero, p.minus_zero), rs = pair2(p.r_scale, p.r_scale);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const uint4 gv = !p.g ? make_uint4(0, 0, 0, 0) : kLate ? gates(v) : g[v];
        const uint4 wv = !p.wp ? make_uint4(0, 0, 0, 0) : kLate ? weights(p.wp, v) : a[v];
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const uint32_t xw = word(x[v], k), rw = word(r[v], k);
            float f0 = 0.f, f1 = 0.f;
            if (p.g) {
                fma_pair(xw, word(gv, k), f0, f1);
            } else {
                f0 = bf16_lo(xw);
                f1 = bf16_hi(xw);
            }
            if (p.wp) {
                const float2 w = add_pair(word(wv, k), p.off);
                f0 *= w.x;
                f1 *= w.y;
            }
            // Each product is rounded and then the sum (a product is a multiply-add to a -0 that comes with the call, or
            // the assembler would join one with the sum): a scale like 0.22 is off by up to 2^-25 in fp32, which its
            // rounded product with a value of few bits is not, and where the exact sum lies between two BF16 values, or
            // is 0, that decides.
            const float2 v2 = unpair(add2(fma2(pair2(f0, f1), pair2(c, c), zero),
                                          fma2(pair2(bf16_lo(rw), bf16_hi(rw)), rs, zero)));
            h[k] = bf16_pack(v2.x, v2.y);
        }
        const int64_t i = first(v);
        if constexpr (kOdd) {  // what is not the row's counts for nothing, whatever the scales make of it
#pragma unroll
            for (int k = 0; k < 4; k++)
                h[k] &= (i + 2 * k >= 0 && i + 2 * k < p.d ? 0xffffu : 0u) |
                        (i + 2 * k + 1 >= 0 && i + 2 * k + 1 < p.d ? 0xffff0000u : 0u);
        } else if (i >= p.d) {
            h[0] = h[1] = h[2] = h[3] = 0;
        }
        if (p.h)
            store8<kOdd>(p.h + row * p.hs, i, p.d, h);
#pragma unroll
        for (int k = 0; k < 4; k++)
            fma_pair(h[k], h[k], s0, s1);
        x[v] = make_uint4(h[0], h[1], h[2], h[3]);
    }
    if (!p.y)
        return;
    if constexpr (!kLate) {
#pragma unroll
        for (int v = 0; v < V; v++)
            a[v] = weights(p.w, v);
    }
    const float ss = kWarp ? warp_sum(s0 + s1) : cta_reduce<false>(s0 + s1, slots + 32);
    const float rstd = rsqrtf(ss / float(p.d) + p.eps);
    float top = 0.f, f[k8 ? V : 1][8];
#pragma unroll
    for (int v = 0; v < V; v++) {
        const uint4 wv = kLate ? weights(p.w, v) : a[v];
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const uint32_t hw = word(x[v], k);
            const float2 w = add_pair(word(wv, k), p.off);
            const float u0 = bf16_lo(hw) * w.x, u1 = bf16_hi(hw) * w.y;
            if constexpr (k8) {
                f[v][2 * k] = u0;
                f[v][2 * k + 1] = u1;
                top = max_nan(top, max_nan(fabsf(u0), fabsf(u1)));
            } else {
                y[k] = bf16_pack(u0 * rstd, u1 * rstd);
            }
        }
        if constexpr (!k8)
            store8<kOdd>(static_cast<uint16_t *>(p.y) + row * p.ys, first(v), p.d, y);
    }
    if constexpr (k8) {
        const RowScale s(kWarp ? warp_max(top) : cta_reduce<true>(top, slots + 64), rstd);
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
__global__ void __launch_bounds__(256) block_warp_kernel(const BlockParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row < p.n)
        block_row<V, k8, true, kOdd>(p, row, threadIdx.x & 31, 32, nullptr);
}

// kLate: weights and gate are loaded where they are used.  (Rows of 16384 that begin anywhere lie on up to
// 2049 steps: 513 threads.)
template <int V, bool k8, bool kOdd, bool kLate, int kMost, int kCtas>
__global__ void __launch_bounds__(kMost, kCtas) block_cta_kernel(const BlockParams p) {
    __shared__ float slots[96];
    grid_dep_launch();
    grid_dep_wait();
    block_row<V, k8, false, kOdd, kLate>(p, blockIdx.x, threadIdx.x, blockDim.x, slots);
}

// Rows of any kind, value by value.
template <bool k8>
__global__ void __launch_bounds__(512) block_any_kernel(const BlockParams p) {
    __shared__ float slots[96];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t row = blockIdx.x;
    const uint16_t *const x = p.x + row * p.xs, *const r = p.r + row * p.rs;
    const uint16_t *const g = p.g ? p.g + row * p.gs : nullptr;
    uint16_t *const h = p.h ? p.h + row * p.hs : nullptr;
    float c = p.b_scale;
    if (p.wp) {
        float ss = 0.f;
        for (int64_t i = threadIdx.x; i < p.d; i += blockDim.x) {
            const float f = bf16_lo(x[i]);
            ss = fmaf(f, f, ss);
        }
        c *= rsqrtf(cta_reduce<false>(ss, slots) / float(p.d) + p.eps);
    }
    auto made = [&](int64_t i) {
        float f = bf16_lo(x[i]);
        if (g)
            f *= bf16_lo(g[i]);
        if (p.wp)
            f *= bf16_lo(p.wp[i]) + p.off;
        return __bfloat16_as_ushort(
            __float2bfloat16_rn(__fadd_rn(__fmul_rn(f, c), __fmul_rn(p.r_scale, bf16_lo(r[i])))));
    };
    float ss = 0.f;
    for (int64_t i = threadIdx.x; i < p.d; i += blockDim.x) {
        const uint16_t b = made(i);
        if (h)
            h[i] = b;
        const float f = bf16_lo(b);
        ss = fmaf(f, f, ss);
    }
    if (!p.y)
        return;
    // from here on x or r may lie under h: what was written is read back
    auto value = [&](int64_t i) { return bf16_lo(h ? h[i] : made(i)); };
    const float rstd = rsqrtf(cta_reduce<false>(ss, slots + 32) / float(p.d) + p.eps);
    float top = 0.f;
    if constexpr (k8) {
        for (int64_t i = threadIdx.x; i < p.d; i += blockDim.x)
            top = max_nan(top, fabsf(value(i) * (bf16_lo(p.w[i]) + p.off)));
        top = cta_reduce<true>(top, slots + 64);
    }
    const RowScale s(top, rstd);
    if (k8 && threadIdx.x == 0)
        p.scale[row] = s.scale;
    for (int64_t i = threadIdx.x; i < p.d; i += blockDim.x) {
        const float u = value(i) * (bf16_lo(p.w[i]) + p.off);
        if constexpr (k8)
            static_cast<uint8_t *>(p.y)[row * p.ys + i] = to_e4m3(s.of(u));
        else
            static_cast<uint16_t *>(p.y)[row * p.ys + i] = __bfloat16_as_ushort(__float2bfloat16_rn(u * rstd));
    }
}

template <bool k8, bool kOdd>
cudaError_t launch_rows(const BlockParams &p, cudaStream_t st) {
    const int vecs = int((p.d + (kOdd ? 14 : 7)) / 8);  // vectors of a row, wherever it begins
    if (vecs <= kWarpDim / 8) {
        const dim3 grid(unsigned((p.n + 7) / 8)), block(256);
        if (vecs <= 32)
            return launch_overlapped(block_warp_kernel<1, k8, kOdd>, grid, block, 0, st, p);
        if (vecs <= 64)
            return launch_overlapped(block_warp_kernel<2, k8, kOdd>, grid, block, 0, st, p);
        return launch_overlapped(block_warp_kernel<4, k8, kOdd>, grid, block, 0, st, p);
    }
    const dim3 grid(static_cast<unsigned>(p.n));
    auto run = [&](auto kernel, int V) {
        return launch_overlapped(kernel, grid, dim3((vecs + 32 * V - 1) / (32 * V) * 32), 0, st, p);
    };
    if constexpr (kOdd) {
        return vecs <= 1088 ? run(block_cta_kernel<2, k8, true, true, 544, 2>, 2)
                            : run(block_cta_kernel<4, k8, true, true, 544, 1>, 4);
    } else {
        // Up to two rows an SM: as many threads as a row has steps (257 x 5120 to 8 bits 3.9 us, half as many
        // 4.4, a quarter 6.5).  More: what keeps the most loads on their way, by CTAs of an SM and registers
        // (8191 x 4096 42.4 us with 5 CTAs of 256 threads, 45.4 with 4; 4000 x 8192 43.5 with 3 of 512, 42.4 with 4 of 256
        // and twice the steps a thread, 56.8 when values were converted one by one; 2000 x 16384 45.3 with 2, with one and
        // early weights 59.8).
        if (vecs <= 1024 && p.n <= 2 * sm_count())
            return run(block_cta_kernel<1, k8, false, false, 1024, 1>, 1);
        if (vecs <= 512)
            return run(block_cta_kernel<2, k8, false, false, 256, 5>, 2);
        if (vecs <= 1024)
            return run(block_cta_kernel<2, k8, false, true, 512, 3>, 2);
        return run(block_cta_kernel<4, k8, false, true, 512, 2>, 4);
    }
}

template <bool k8>
cudaError_t launch_block(const BlockParams &p, bool vec, bool alike, cudaStream_t st) {
    if (p.d > kMaxVecDim || !alike)
        return launch_overlapped(block_any_kernel<k8>, dim3(unsigned(p.n)), dim3(512), 0, st, p);
    return vec ? launch_rows<k8, false>(p, st) : launch_rows<k8, true>(p, st);
}

uintptr_t bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }

uw_status run_block(const uw_block *b, const uint16_t *x, int64_t xs, const uint16_t *r, int64_t rs, uint16_t *h,
                    int64_t hs, const uint16_t *w, int64_t n, int64_t d, void *y, int64_t ys, float *scale, bool k8,
                    void *stream) {
    if (!b || n < 0 || !(b->eps >= 0.f) || !std::isfinite(b->weight_offset) || !std::isfinite(b->residual_scale) ||
        !std::isfinite(b->block_scale))
        return UW_ERR_INVALID_ARG;
    // no rows need no buffers (those of empty tensors are null)
    if (n != 0 && (!x || !r || !w != !y || (!y && (!h || k8)) || (k8 && !scale)))
        return UW_ERR_INVALID_ARG;
    if (d <= 0)
        return UW_ERR_SHAPE;
    if (n > 0x7fffffff || d > 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    const uint16_t *const g = b->gate_dev;
    const int64_t gs = g && b->gate_stride ? b->gate_stride : 0;
    if ((n > 1 && (xs < d || rs < d || (y && ys < d) || (h && hs < d))) || gs < 0 || (gs && n > 1 && gs < d))
        return UW_ERR_INVALID_ARG;
    if (n == 0)
        return UW_OK;
    if (((bits(x) | bits(r) | bits(h) | bits(w) | bits(g) | bits(b->post_weight_dev)) & 1) || (!k8 && (bits(y) & 1)) ||
        (k8 && (bits(scale) & 3)))
        return UW_ERR_INVALID_ARG;
    // where a tensor's rows begin, in values: eight of them are 16 bytes (8 of e4m3)
    const uint64_t x0 = bits(x) / 2;
    auto as_x = [&](uint64_t first, int64_t stride) {
        return (first - x0) % 8 == 0 && (n == 1 || (stride - xs) % 8 == 0);
    };
    const bool alike = as_x(bits(r) / 2, rs) && (!y || as_x(bits(y) / (k8 ? 1 : 2), ys)) &&
                       (!h || as_x(bits(h) / 2, hs)) && (!gs || as_x(bits(g) / 2, gs));
    // (what is not given is null and on every step)
    const bool vec = d % 8 == 0 && x0 % 8 == 0 && (n == 1 || xs % 8 == 0) &&
                     ((bits(w) | bits(b->post_weight_dev) | (gs ? 0 : bits(g))) & 15) == 0;
    const BlockParams p{x,  r,  g,  b->post_weight_dev, w, h, y, scale, xs, rs, gs, hs, ys, n, d, b->eps,
                        b->weight_offset, b->residual_scale, b->block_scale, -0.f};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (k8 ? launch_block<true>(p, vec, alike, st) : launch_block<false>(p, vec, alike, st)) == cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}

}  // namespace
}  // namespace uw

extern "C" uw_status uw_block_norm(const uw_block *b, const uint16_t *x, int64_t xs, const uint16_t *r, int64_t rs,
                                   uint16_t *h, int64_t hs, const uint16_t *w, int64_t n, int64_t d, uint16_t *y,
                                   int64_t ys, void *stream) {
    return uw::run_block(b, x, xs, r, rs, h, hs, w, n, d, y, ys, nullptr, false, stream);
}

extern "C" uw_status uw_block_norm_e4m3(const uw_block *b, const uint16_t *x, int64_t xs, const uint16_t *r,
                                        int64_t rs, uint16_t *h, int64_t hs, const uint16_t *w, int64_t n, int64_t d,
                                        uint8_t *q, int64_t qs, float *scale, void *stream) {
    return uw::run_block(b, x, xs, r, rs, h, hs, w, n, d, q, qs, scale, true, stream);
}
