// Into the 4-bit paged cache and back.
//   append  rotates q and k by their positions, quantises k and v vector by
//           vector (one token, one kv head) and writes codes and params
//   read    the new tokens' entries as BF16
//
// Both move little per token (48 vectors of 256 bytes for 32 + 2 x 8 heads of
// 128), so they are bound by latency for a decode step and by memory for
// prompts.  A vector belongs to D / 8 lanes, 16 bytes each; a warp takes
// 32 / (D / 8) heads of one token at a time, `chunk` times, so that the
// token's place and its row of the rotation table are found once for all of
// them.  Minimum and maximum are joined by shuffles within the vector's lanes.
//
// The rotation rounds each product and the sum (no fused multiply-add), so
// that the same inputs give the same codes as the formula computed step by
// step in fp32; a code is a step function, and a last-bit difference before
// it could show as a whole step after it.
#include "kernels.h"
#include "kv4.cuh"
#include "kv4_host.h"

namespace uw {

namespace {

struct AppendParams {
    Kv4View v;
    Rows q, qo, k, vv;
    const float *cos, *sin;
    int64_t rope_len;
    int32_t q_heads, rot, interleaved, chunk;
};

template <int D>
__device__ __forceinline__ float vec_min(float x) {
#pragma unroll
    for (int o = D / 16; o; o >>= 1)
        x = fminf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// Codes and params of eight values of a vector of D, whose lanes are
// together; all 32 lanes call.  Returns the lane's eight codes.
template <int D>
__device__ __forceinline__ uint32_t quantise(const float (&f)[8], uint32_t *params) {
    float lo = f[0], hi = f[0];
    bool finite = true;
#pragma unroll
    for (int k = 0; k < 8; k++) {
        lo = fminf(lo, f[k]);
        hi = fmaxf(hi, f[k]);
        finite = finite && fabsf(f[k]) <= 3.4e38f;
    }
    lo = vec_min<D>(lo);
    hi = -vec_min<D>(-hi);
    const float bad = -vec_min<D>(finite ? 0.f : -1.f);
    if (bad > 0.f) {
        *params = 0x7fc07fc0u;
        return 0u;
    }
    // halves: hi - lo of two finite values may not be finite
    const float lo2 = 0.5f * lo;
    const uint32_t sb = bf16_pack((0.5f * hi - lo2) / 7.5f, lo);
    const float s2 = 0.5f * bf16_lo(sb);
    *params = sb;
    uint32_t codes = 0u;
#pragma unroll
    for (int k = 0; k < 8; k++) {
        const float c = s2 > 0.f ? rintf((0.5f * f[k] - lo2) / s2) : 0.f;
        codes |= uint32_t(fminf(fmaxf(c, 0.f), 15.f)) << (4 * k);
    }
    return codes;
}

template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const AppendParams p) {
    constexpr int L = D / 8;       // lanes of a vector
    constexpr int G = 32 / L;      // vectors a warp takes at once
    grid_dep_launch();
    grid_dep_wait();
    const Kv4View &v = p.v;
    const int lane = threadIdx.x & 31, c = lane % L;
    const int total = p.q_heads + 2 * v.heads;
    const int per_token = (total + G * p.chunk - 1) / (G * p.chunk);
    const int64_t unit = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = unit / per_token;
    if (t >= v.n_tokens)
        return;
    const int s = kv4_find_seq(v, int(t));
    const Seq q = kv4_seq(v, s);
    if (t < q.t0 || t >= int64_t(q.t0) + q.n)
        return;  // a token of no sequence
    const int32_t pos = q.len - q.n + (int32_t(t) - q.t0);
    if (pos < 0 || (p.rot && pos >= p.rope_len)) {
        if (lane == 0)
            atomicOr(v.status, uint32_t(kStatusBadCache));
        return;
    }
    // The lane's share of the rotation: its eight values are one side of
    // eight pairs (half split: the partner's lie rot / 2 values on or back),
    // or four whole pairs (interleaved).
    const int half = p.rot / 2, i0 = 8 * c;
    const bool rotated = i0 < p.rot, second = !p.interleaved && i0 >= half;
    float cs[8], sn[8];
    if (rotated) {
        const int64_t row = int64_t(pos) * half;
        if (p.interleaved) {
#pragma unroll
            for (int k = 0; k < 4; k++) {
                cs[k] = __ldg(p.cos + row + 4 * c + k);
                sn[k] = __ldg(p.sin + row + 4 * c + k);
            }
        } else {
            const int j = second ? i0 - half : i0;
#pragma unroll
            for (int k = 0; k < 8; k++) {
                cs[k] = __ldg(p.cos + row + j + k);
                sn[k] = __ldg(p.sin + row + j + k);
            }
        }
    }
    const int partner = p.interleaved || !rotated ? lane : second ? lane - half / 8 : lane + half / 8;
    const int slot = pos & ((1 << v.page_log2) - 1);

    const int h0 = int(unit - t * per_token) * G * p.chunk + lane / L;
    for (int ci = 0; ci < p.chunk; ci++) {
        const int h = h0 + ci * G;
        const bool mine = h < total;
        // q heads first, then k, then v
        const int kind = h < p.q_heads ? 0 : h < p.q_heads + v.heads ? 1 : 2;
        const int hk = kind == 0 ? h : kind == 1 ? h - p.q_heads : h - p.q_heads - v.heads;
        const Rows &src = kind == 0 ? p.q : kind == 1 ? p.k : p.vv;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (mine)
            x = *reinterpret_cast<const uint4 *>(src.p + t * src.ts + hk * src.hs + i0);
        uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4];
#pragma unroll
        for (int k = 0; k < 4; k++)
            b[k] = __shfl_sync(0xffffffffu, a[k], partner);
        if (kind != 2 && rotated) {
            if (p.interleaved) {
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float u = bf16_lo(a[k]), w = bf16_hi(a[k]);
                    a[k] = bf16_pack(__fsub_rn(__fmul_rn(u, cs[k]), __fmul_rn(w, sn[k])),
                                     __fadd_rn(__fmul_rn(w, cs[k]), __fmul_rn(u, sn[k])));
                }
            } else {
                // first side: a c - b s; second side: a c + b s (a its own value, b the partner's)
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float s0 = second ? sn[2 * k] : -sn[2 * k], s1 = second ? sn[2 * k + 1] : -sn[2 * k + 1];
                    a[k] = bf16_pack(__fadd_rn(__fmul_rn(bf16_lo(a[k]), cs[2 * k]), __fmul_rn(bf16_lo(b[k]), s0)),
                                     __fadd_rn(__fmul_rn(bf16_hi(a[k]), cs[2 * k + 1]), __fmul_rn(bf16_hi(b[k]), s1)));
                }
            }
        }
        if (kind == 0 && mine)
            *reinterpret_cast<uint4 *>(p.qo.p + t * p.qo.ts + hk * p.qo.hs + i0) = make_uint4(a[0], a[1], a[2], a[3]);
        if (__ballot_sync(0xffffffffu, mine && kind != 0)) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                f[2 * k] = bf16_lo(a[k]);
                f[2 * k + 1] = bf16_hi(a[k]);
            }
            uint32_t params;
            const uint32_t codes = quantise<D>(f, &params);
            if (mine && kind != 0) {
                uint8_t *blk = kv4_block<D>(v, s, pos, hk);
                if (blk) {
                    const int is_v = kind == 2;
                    *reinterpret_cast<uint32_t *>(blk + kv4_codes<D>(v.page_log2, slot, is_v) + 4 * c) = codes;
                    if (c == 0)
                        *reinterpret_cast<uint32_t *>(blk + kv4_params<D>(v.page_log2, slot, is_v)) = params;
                }
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4View v, const Rows ko, const Rows vo, const int chunk) {
    constexpr int L = D / 8, G = 32 / L;
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, c = lane % L;
    const int total = 2 * v.heads;
    const int per_token = (total + G * chunk - 1) / (G * chunk);
    const int64_t unit = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = unit / per_token;
    if (t >= v.n_tokens)
        return;
    const int s = kv4_find_seq(v, int(t));
    const Seq q = kv4_seq(v, s);
    if (t < q.t0 || t >= int64_t(q.t0) + q.n)
        return;
    const int32_t pos = q.len - q.n + (int32_t(t) - q.t0);
    if (pos < 0) {
        if (lane == 0)
            atomicOr(v.status, uint32_t(kStatusBadCache));
        return;
    }
    const int slot = pos & ((1 << v.page_log2) - 1);
    const int h0 = int(unit - t * per_token) * G * chunk + lane / L;
    for (int ci = 0; ci < chunk; ci++) {
        const int h = h0 + ci * G;
        if (h >= total)
            break;
        const int is_v = h >= v.heads, hk = is_v ? h - v.heads : h;
        const uint8_t *blk = kv4_block<D>(v, s, pos, hk);
        if (!blk)
            continue;
        const uint32_t codes = *reinterpret_cast<const uint32_t *>(blk + kv4_codes<D>(v.page_log2, slot, is_v) + 4 * c);
        const uint32_t par = *reinterpret_cast<const uint32_t *>(blk + kv4_params<D>(v.page_log2, slot, is_v));
        const float scale = bf16_lo(par), lo = bf16_hi(par);
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; k++)
            o[k] = bf16_pack(fmaf(float((codes >> (8 * k)) & 15u), scale, lo),
                             fmaf(float((codes >> (8 * k + 4)) & 15u), scale, lo));
        const Rows &dst = is_v ? vo : ko;
        *reinterpret_cast<uint4 *>(dst.p + t * dst.ts + hk * dst.hs + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// Heads a warp takes one after the other: enough warps for two per scheduler
// come first, fewer and longer ones after that.
int heads_per_warp(int64_t tokens, int rounds) {
    int chunk = 1;
    while (chunk < rounds && tokens * ((rounds + 2 * chunk - 1) / (2 * chunk)) >= 152 * 4 * 2)
        chunk *= 2;
    return chunk;
}

}  // namespace
}  // namespace uw

using namespace uw;

extern "C" uw_status uw_kv4_append(const uw_kv4_cache *c, const int32_t *start, const int32_t *len, int64_t n_tokens,
                                   const uw_kv4_rows *q, int32_t q_heads, const uw_kv4_rows *q_out,
                                   const uw_kv4_rows *k, const uw_kv4_rows *v, const float *cos, const float *sin,
                                   int64_t rope_len, int32_t rot_dim, int32_t interleaved, void *ws, size_t ws_bytes,
                                   void *stream) {
    AppendParams p{};
    uw_status s = kv4_view(c, start, len, n_tokens, ws, ws_bytes, &p.v);
    if (s != UW_OK)
        return s;
    if (q_heads < 0 || (q_heads > 0) != (q != nullptr) || (q_heads > 0) != (q_out != nullptr) || !k || !v ||
        rot_dim < 0 || rope_len < 0 || (rot_dim > 0 && (!cos || !sin)))
        return UW_ERR_INVALID_ARG;
    if (rot_dim % 16 || rot_dim > c->head_dim || q_heads > kKv4MaxHeads)
        return UW_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) & 3)
        return UW_ERR_INVALID_ARG;
    if (p.v.n_tokens == 0)
        return UW_OK;
    if (!kv4_rows(k, &p.k) || !kv4_rows(v, &p.vv) || (q && (!kv4_rows(q, &p.q) || !kv4_rows(q_out, &p.qo))))
        return UW_ERR_INVALID_ARG;
    p.cos = cos;
    p.sin = sin;
    p.rope_len = rope_len;
    p.q_heads = q_heads;
    p.rot = rot_dim;
    p.interleaved = interleaved != 0;
    const int g = c->head_dim == 128 ? 2 : 4, rounds = (q_heads + 2 * c->kv_heads + g - 1) / g;
    p.chunk = heads_per_warp(n_tokens, rounds);
    const int64_t units = n_tokens * ((rounds + p.chunk - 1) / p.chunk);
    if (units > int64_t(8) * 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    const dim3 grid(unsigned((units + 7) / 8));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (c->head_dim == 128 ? launch_overlapped(kv4_append_kernel<128>, grid, dim3(256), 0, st, p)
                               : launch_overlapped(kv4_append_kernel<64>, grid, dim3(256), 0, st, p)) == cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}

extern "C" uw_status uw_kv4_read(const uw_kv4_cache *c, const int32_t *start, const int32_t *len, int64_t n_tokens,
                                 const uw_kv4_rows *k, const uw_kv4_rows *v, void *ws, size_t ws_bytes, void *stream) {
    Kv4View view{};
    uw_status s = kv4_view(c, start, len, n_tokens, ws, ws_bytes, &view);
    if (s != UW_OK)
        return s;
    Rows ko, vo;
    if (!k || !v)
        return UW_ERR_INVALID_ARG;
    if (view.n_tokens == 0)
        return UW_OK;
    if (!kv4_rows(k, &ko) || !kv4_rows(v, &vo))
        return UW_ERR_INVALID_ARG;
    const int g = c->head_dim == 128 ? 2 : 4, rounds = (2 * c->kv_heads + g - 1) / g;
    const int chunk = heads_per_warp(n_tokens, rounds);
    const int64_t units = n_tokens * ((rounds + chunk - 1) / chunk);
    if (units > int64_t(8) * 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    const dim3 grid(unsigned((units + 7) / 8));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (c->head_dim == 128 ? launch_overlapped(kv4_read_kernel<128>, grid, dim3(256), 0, st, view, ko, vo, chunk)
                               : launch_overlapped(kv4_read_kernel<64>, grid, dim3(256), 0, st, view, ko, vo, chunk)) ==
                   cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}
