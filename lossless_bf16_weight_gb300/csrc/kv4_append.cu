// Into the 4-bit paged cache and back.
//   append  rotates q and k by their positions, quantises k and v vector by
//           vector (one token, one kv head) and writes codes and params
//   read    the new tokens' entries as BF16
//
// A decode step moves little (48 vectors of 256 bytes a token for 32 + 2 x 8
// heads of 128): its time is latency.  For prompts it is loads in flight: issue
// slots are 64% used, memory runs at 0.67 of a copy, and four CTAs of 64 registers a
// thread are what an SM holds.  A vector belongs to D / 8 lanes, 16 bytes each; a warp takes q heads
// of one token, or k and v heads, 32 / (D / 8) at a time, and finds the token's
// place and its row of the rotation table once for all of them, while the
// first vectors are on their way.  Minimum and maximum are joined by shuffles
// within the vector's lanes.
//
// Measured, 32 query and 8 kv heads of 128: append 1 token 2.3 us, 64 tokens 3.3,
// 8143 tokens 40 us (4.4 TB/s); read 1.7, 2.2 and 10.5 us (4.0 TB/s).  With positions on three axes
// and k in BF16 beside the codes: 3.6, 4.3 and 43.6 us (4.5 TB/s; pairs of four that turn by several axes 47).
//
// The rotation rounds each product and the sum (no fused multiply-add), and the
// quotient of the quantisation is correctly rounded, so that the same inputs
// give the same codes as the formula computed step by step in fp32; a code is a
// step function, and a last-bit difference before it could show as a whole step
// after it.
#include <type_traits>

#include "kernels.h"
#include "kv4.cuh"
#include "kv4_host.h"
#include "rope.cuh"

namespace uw {

namespace {

struct AppendParams {
    Kv4View v;
    Rows q, qo, k, vv;
    const float *cos, *sin;
    int64_t rope_len;
    int32_t q_heads, rot, interleaved;
    int32_t q_units, kv_units;    // warps a token: of q heads, and of k and v heads
    int32_t q_rounds, kv_rounds;  // heads such a warp takes one after the other (times 32 / (D / 8))
    float minus_zero;             // -0, which the compiler does not know (rotate())
    // positions on several axes (kAxes): each token's, and the rotated k in BF16, if wanted
    Axes axes;
    RopePlan plan;  // of q
    Rows ko;
};

// Vectors a lane has on their way (8143 and 64 tokens: 2 41.8 and 3.3 us, 4 41.8 and 4.4, 1 45.8 and 3.3).
constexpr int kAhead = 2;

// Smaller halves of two pairs of BF16; NaN wherever one is.
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// a / b correctly rounded (two quotients at once), from -b and r = 1 / b correctly rounded: two corrections
// of a r by its remainder (Markstein, IBM J. Res. Dev. 34, 1990).  For the
// quotients of quantise(), 0 .. 16 or so, with neither b nor r near the ends of
// fp32's range.
__device__ __forceinline__ uint64_t divide_by(uint64_t a, uint64_t minus_b, uint64_t r) {
    uint64_t q = mul2(a, r);
    q = fma2(fma2(q, minus_b, a), r, q);
    return fma2(fma2(q, minus_b, a), r, q);
}

// Codes and params of eight values (pairs of BF16) of a vector of D, whose lanes
// are together; all 32 lanes call.  Returns the lane's eight codes.
template <int D>
__device__ __forceinline__ uint32_t quantise(const uint32_t (&x)[4], uint32_t *params) {
    constexpr uint32_t kSigns = 0x80008000u;
    // (smallest value, largest with its sign turned) as a pair
    const uint32_t l = min2(min2(x[0], x[1]), min2(x[2], x[3]));
    const uint32_t h = min2(min2(x[0] ^ kSigns, x[1] ^ kSigns), min2(x[2] ^ kSigns, x[3] ^ kSigns));
    uint32_t ends = min2(__byte_perm(l, h, 0x5410), __byte_perm(l, h, 0x7632));
#pragma unroll
    for (int o = D / 16; o; o >>= 1)
        ends = min2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
    const float lo = bf16_lo(ends), hi = -bf16_hi(ends);
    // halves: hi - lo of two finite values may not be finite
    const float lo2 = 0.5f * lo, range2 = 0.5f * hi - lo2;
    if (!(range2 <= 3.4e38f)) {  // a value that is not finite
        *params = 0x7fc07fc0u;
        return 0u;
    }
    const uint32_t sb = bf16_pack(range2 / 7.5f, lo);
    const float s2 = 0.5f * bf16_lo(sb);
    *params = sb;
    if (!(s2 > 0.f))
        return 0u;
    uint32_t codes = 0u;
    if (s2 > 1e-30f && s2 < 1e30f) {
        // Quotients from 0 to 15.06 (the scale is within 2^-8 of its value), so no
        // clamping; the integer they round to is read off the sum with 1.5 * 2^23.
        constexpr float kRound = 12582912.f;
        const float rcp = __frcp_rn(s2);
        const uint64_t r = pair2(rcp, rcp), minus_s2 = pair2(-s2, -s2), minus_lo2 = pair2(-lo2, -lo2);
        const uint64_t a_half = pair2(0.5f, 0.5f), round = pair2(kRound, kRound);
        constexpr uint32_t kOff = 0x4B400000u * 0x11111111u;  // the sums' other bits, as they add up
#pragma unroll
        for (int k = 3; k >= 0; k--) {
            const uint64_t f = fma2(a_half, pair2(bf16_lo(x[k]), bf16_hi(x[k])), minus_lo2);
            const float2 n = unpair(add2(divide_by(f, minus_s2, r), round));
            codes = (codes * 16u + __float_as_uint(n.y)) * 16u + __float_as_uint(n.x);
        }
        codes -= kOff;
    } else {
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const float f = k & 1 ? bf16_hi(x[k / 2]) : bf16_lo(x[k / 2]);
            codes |= uint32_t(fminf(fmaxf(rintf((0.5f * f - lo2) / s2), 0.f), 15.f)) << (4 * k);
        }
    }
    return codes;
}

// kAxes: a pair turns by its token's position on the pair's axis, not by the
// place in the sequence, and k_out, if there is one, takes the rotated k.
template <int D, bool kAxes>
__global__ void __launch_bounds__(256, 4) kv4_append_kernel(const AppendParams p) {
    constexpr int L = D / 8;       // lanes of a vector
    constexpr int G = 32 / L;      // vectors a warp takes at once
    grid_dep_launch();
    grid_dep_wait();
    const Kv4View &v = p.v;
    const int lane = threadIdx.x & 31, c = lane % L;
    const uint32_t per_token = uint32_t(p.q_units + p.kv_units);
    const uint64_t unit = uint64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = (unit >> 32) ? unit / per_token : uint32_t(unit) / per_token;
    if (t >= v.n_tokens)
        return;
    const int part = int(unit - uint64_t(t) * per_token);
    // The unit's vectors: q heads, or k heads and then v heads.  They are loaded
    // before the token is looked up, a group of kAhead at a time, and with them the
    // other sides of their pairs (the same cache lines), before anything is
    // written: q_out may be q.
    const bool of_q = part < p.q_units;
    if (kAxes && p.rot && of_q) {  // both sides of a pair by one lane
        const int first = part * p.plan.rounds * p.plan.per;
        auto rotated = [&](auto interleaved) {
            rope_heads<decltype(interleaved)::value>(
                p.plan, p.axes, p.cos, p.sin, pair2(p.minus_zero, p.minus_zero), first, p.q_heads,
                [&](int j) { return p.q.p + t * p.q.ts + j * p.q.hs; },
                [&](int j) { return p.qo.p + t * p.qo.ts + j * p.qo.hs; }, [&](AxesAt &turn) {
                    const bool found = turn.find(p.axes, t, p.rope_len);
                    const Seq q = kv4_seq(v, kv4_find_seq(v, int(t)));
                    if (t < q.t0 || t >= int64_t(q.t0) + q.n)
                        return false;  // a token of no sequence
                    if (found && q.len - q.n + (int32_t(t) - q.t0) >= 0)
                        return true;
                    if (lane == 0)
                        atomicOr(v.status, kStatusBadCache);
                    return false;
                });
        };
        if (p.interleaved)
            rotated(std::true_type());
        else
            rotated(std::false_type());
        return;
    }
    const int rounds = of_q ? p.q_rounds : p.kv_rounds, all = of_q ? p.q_heads : 2 * v.heads;
    const int j0 = (of_q ? part : part - p.q_units) * rounds * G + lane / L;
    const int half = p.rot / 2, i0 = 8 * c;
    Rotation r;
    r.on = i0 < p.rot;
    r.interleaved = p.interleaved;
    const bool second = i0 >= half;
    const int other = second ? -half : half;  // half split: where the other side's values are, from the own
    uint4 x[kAhead], o[kAhead];
    auto fetch = [&](int n0) {
#pragma unroll
        for (int n = 0; n < kAhead; n++) {
            const int j = j0 + (n0 + n) * G;
            const bool in = n0 + n < rounds && j < all, is_v = !of_q && j >= v.heads;
            const Rows &src = of_q ? p.q : is_v ? p.vv : p.k;
            const uint16_t *at = src.p + t * src.ts + (is_v ? j - v.heads : j) * src.hs + i0;
            x[n] = in ? *reinterpret_cast<const uint4 *>(at) : make_uint4(0, 0, 0, 0);
            o[n] = in && !is_v && r.on && !r.interleaved ? *reinterpret_cast<const uint4 *>(at + other)
                                                         : make_uint4(0, 0, 0, 0);
        }
    };
    fetch(0);
    // positions on axes and their rows of the tables do not wait for the token's place
    bool found = true;
    if (kAxes && p.rot) {
        AxesAt turn;
        found = turn.find(p.axes, t, p.rope_len);
        if (found && r.on) {
            const int j = p.interleaved ? 4 * c : second ? i0 - half : i0;
            const float4 c0 = turn.four(p.axes, p.cos, half, j), s0 = turn.four(p.axes, p.sin, half, j);
            if (p.interleaved) {
                r.of_pairs(c0, s0);
            } else {
                r.of_side(c0, s0, 0, second);
                r.of_side(turn.four(p.axes, p.cos, half, j + 4), turn.four(p.axes, p.sin, half, j + 4), 1, second);
            }
        }
    }
    const int s = kv4_find_seq(v, int(t));
    const Seq q = kv4_seq(v, s);
    if (t < q.t0 || t >= int64_t(q.t0) + q.n)
        return;  // a token of no sequence
    const int32_t pos = q.len - q.n + (int32_t(t) - q.t0);
    if (pos < 0 || !found || (!kAxes && p.rot && pos >= p.rope_len)) {
        if (lane == 0)
            atomicOr(v.status, kStatusBadCache);
        return;
    }
    if (!kAxes && r.on) {
        const int64_t row = int64_t(pos) * half;
        if (p.interleaved) {
            r.of_pairs(*reinterpret_cast<const float4 *>(p.cos + row + 4 * c),
                       *reinterpret_cast<const float4 *>(p.sin + row + 4 * c));
        } else {
            const int j = second ? i0 - half : i0;
#pragma unroll
            for (int k = 0; k < 2; k++)
                r.of_side(*reinterpret_cast<const float4 *>(p.cos + row + j + 4 * k),
                          *reinterpret_cast<const float4 *>(p.sin + row + j + 4 * k), k, second);
        }
    }

    const uint64_t zero = pair2(p.minus_zero, p.minus_zero);
    if (of_q) {
        uint16_t *const dst = p.qo.p + t * p.qo.ts + j0 * p.qo.hs + i0;
        for (int n0 = 0;;) {
            __syncwarp();
#pragma unroll
            for (int n = 0; n < kAhead; n++) {
                uint32_t a[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
                rotate(r, zero, a, o[n]);
                if (n0 + n < rounds && j0 + (n0 + n) * G < all)
                    *reinterpret_cast<uint4 *>(dst + int64_t(n0 + n) * G * p.qo.hs) =
                        make_uint4(a[0], a[1], a[2], a[3]);
            }
            n0 += kAhead;
            if (n0 >= rounds)
                return;
            fetch(n0);
        }
    }
    uint8_t *const page = kv4_block<D>(v, s, pos, 0);  // the token's page, block of head 0
    if (!page && !(kAxes && p.ko.p))
        return;
    const int slot = pos & ((1 << v.page_log2) - 1);
    const int64_t block = int64_t(D + 8) << v.page_log2;
    for (int n0 = 0;;) {
        if constexpr (kAxes)
            __syncwarp();  // k_out may be k
#pragma unroll
        for (int n = 0; n < kAhead; n++) {
            const int j = j0 + (n0 + n) * G;
            if (n0 + n >= rounds || j - lane / L >= all)
                return;
            const bool is_v = j >= v.heads;
            uint32_t a[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
            if (!is_v)
                rotate(r, zero, a, o[n]);
            if (kAxes && p.ko.p && !is_v)
                *reinterpret_cast<uint4 *>(p.ko.p + t * p.ko.ts + j * p.ko.hs + i0) =
                    make_uint4(a[0], a[1], a[2], a[3]);
            uint32_t params;
            const uint32_t codes = quantise<D>(a, &params);
            if (j < all && (!kAxes || page)) {
                uint8_t *const blk = page + (is_v ? j - v.heads : j) * block;
                *reinterpret_cast<uint32_t *>(blk + kv4_codes<D>(v.page_log2, slot, is_v) + 4 * c) = codes;
                if (c == 0)
                    *reinterpret_cast<uint32_t *>(blk + kv4_params<D>(v.page_log2, slot, is_v)) = params;
            }
        }
        n0 += kAhead;
        if (n0 >= rounds)
            return;
        fetch(n0);
    }
}

// Ahead: vectors a lane has on their way, as many as it has in all or one (8143 tokens:
// 8 10.5 us, 4 11.4, 2 13.0; one token with 8 1.94 us, with one 1.75).
template <int D, int Ahead>
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
            atomicOr(v.status, kStatusBadCache);
        return;
    }
    const int slot = pos & ((1 << v.page_log2) - 1);
    const uint32_t block = uint32_t(D + 8) << v.page_log2;  // (all heads of a page: below 2^32)
    const uint8_t *const page = kv4_block<D>(v, s, pos, 0);
    if (!page)
        return;
    const int h0 = int(unit - t * per_token) * G * chunk + lane / L;
    uint16_t *const ko_at = ko.p + t * ko.ts + 8 * c, *const vo_at = vo.p + t * vo.ts + 8 * c;
    const uint64_t minus16 = pair2(-16.f, -16.f);
    for (int c0 = 0; c0 < chunk; c0 += Ahead) {
        // all loads before the first store, which could otherwise not pass it
        uint32_t codes[Ahead], par[Ahead];
#pragma unroll
        for (int n = 0; n < Ahead; n++) {
            const int h = h0 + (c0 + n) * G;
            const bool in = c0 + n < chunk && h < total, is_v = h >= v.heads;
            const uint8_t *const blk = page + (is_v ? h - v.heads : h) * block;
            const uint8_t *const code_at = blk + kv4_codes<D>(v.page_log2, slot, is_v) + 4 * c;
            const uint8_t *const par_at = blk + kv4_params<D>(v.page_log2, slot, is_v);
            codes[n] = in ? *reinterpret_cast<const uint32_t *>(code_at) : 0u;
            par[n] = in ? *reinterpret_cast<const uint32_t *>(par_at) : 0u;
        }
#pragma unroll
        for (int n = 0; n < Ahead; n++) {
            const int h = h0 + (c0 + n) * G;
            if (c0 + n >= chunk || h >= total)
                return;
            const uint64_t scale = pair2(bf16_lo(par[n]), bf16_lo(par[n]));
            const uint64_t lo = pair2(bf16_hi(par[n]), bf16_hi(par[n]));
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                // a code at the top of the mantissa of 16 is 16 + c
                auto up = [&](int at) {
                    const uint32_t x = at < 19 ? codes[n] << (19 - at) : codes[n] >> (at - 19);
                    return __uint_as_float((x & 0x780000u) | 0x41800000u);
                };
                const float2 x = unpair(fma2(add2(pair2(up(8 * k), up(8 * k + 4)), minus16), scale, lo));
                o[k] = bf16_pack(x.x, x.y);
            }
            uint16_t *const dst = h >= v.heads ? vo_at + (h - v.heads) * vo.hs : ko_at + h * ko.hs;
            *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Vectors a warp takes one after the other (up to `most`) of the `all` of a token:
// warps for two per scheduler come first, longer ones after that (8143 tokens
// appended in 40 us, with one vector a warp 95; read in 10.5, with two 15).
int rounds_of(int64_t tokens, int all, int most) {
    int n = 1;
    const int64_t two = 2 * 4 * int64_t(sm_count());  // warps, of four schedulers an SM
    while (2 * n <= most && n < all && tokens * ((all + 2 * n - 1) / (2 * n)) >= two)
        n *= 2;
    return n;
}

}  // namespace
}  // namespace uw

using namespace uw;

// Both entry points: axes NULL turns every pair by the token's place.
static uw_status run_append(const uw_kv4_cache *c, const int32_t *start, const int32_t *len, int64_t n_tokens,
                            const uw_kv4_rows *q, int32_t q_heads, const uw_kv4_rows *q_out, const uw_kv4_rows *k,
                            const uw_kv4_rows *v, const float *cos, const float *sin, int64_t rope_len,
                            int32_t rot_dim, int32_t interleaved, const uw_rope *axes, const uw_kv4_rows *k_out,
                            void *ws, size_t ws_bytes, void *stream) {
    AppendParams p{};
    uw_status s = kv4_view(c, start, len, n_tokens, ws, ws_bytes, &p.v);
    if (s != UW_OK)
        return s;
    if (q_heads < 0 || (q_heads > 0) != (q != nullptr) || (q_heads > 0) != (q_out != nullptr) || !k || !v ||
        rot_dim < 0 || rope_len < 0 || (rot_dim > 0 && (!cos || !sin)))
        return UW_ERR_INVALID_ARG;
    if (rot_dim % 16 || rot_dim > c->head_dim || q_heads > kKv4MaxHeads)
        return UW_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) & 15)
        return UW_ERR_INVALID_ARG;
    if (axes && (s = rope_axes_map(*axes, p.v.n_tokens, &p.axes)) != UW_OK)
        return s;
    if (p.v.n_tokens == 0)
        return UW_OK;
    if (!kv4_rows(k, &p.k) || !kv4_rows(v, &p.vv) || (q && (!kv4_rows(q, &p.q) || !kv4_rows(q_out, &p.qo))) ||
        (k_out && !kv4_rows(k_out, &p.ko)))
        return UW_ERR_INVALID_ARG;
    p.cos = cos;
    p.sin = sin;
    p.rope_len = rope_len;
    p.q_heads = q_heads;
    p.rot = rot_dim;
    p.interleaved = interleaved != 0;
    p.minus_zero = -0.f;
    const int g = c->head_dim == 128 ? 2 : 4, q_all = (q_heads + g - 1) / g, kv_all = (2 * c->kv_heads + g - 1) / g;
    p.q_rounds = rounds_of(n_tokens, q_all, 16);
    p.kv_rounds = rounds_of(n_tokens, kv_all, 8);
    p.q_units = (q_all + p.q_rounds - 1) / p.q_rounds;
    p.kv_units = (kv_all + p.kv_rounds - 1) / p.kv_rounds;
    if (axes && rot_dim && q_heads) {
        p.plan = RopePlan(n_tokens, q_heads, rot_dim, c->head_dim, 2 * 4 * int64_t(sm_count()));
        p.q_units = p.plan.units;
    }
    const int64_t units = n_tokens * (p.q_units + p.kv_units);
    if (units > int64_t(8) * 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    const dim3 grid(unsigned((units + 7) / 8));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto run = [&](auto kernel) { return launch_overlapped(kernel, grid, dim3(256), 0, st, p); };
    const cudaError_t e = c->head_dim == 128 ? (axes ? run(kv4_append_kernel<128, true>) : run(kv4_append_kernel<128, false>))
                                             : (axes ? run(kv4_append_kernel<64, true>) : run(kv4_append_kernel<64, false>));
    return e == cudaSuccess ? UW_OK : UW_ERR_CUDA;
}

extern "C" uw_status uw_kv4_append(const uw_kv4_cache *c, const int32_t *start, const int32_t *len, int64_t n_tokens,
                                   const uw_kv4_rows *q, int32_t q_heads, const uw_kv4_rows *q_out,
                                   const uw_kv4_rows *k, const uw_kv4_rows *v, const float *cos, const float *sin,
                                   int64_t rope_len, int32_t rot_dim, int32_t interleaved, void *ws, size_t ws_bytes,
                                   void *stream) {
    return run_append(c, start, len, n_tokens, q, q_heads, q_out, k, v, cos, sin, rope_len, rot_dim, interleaved,
                      nullptr, nullptr, ws, ws_bytes, stream);
}

extern "C" uw_status uw_kv4_append_axes(const uw_kv4_cache *c, const int32_t *start, const int32_t *len,
                                        int64_t n_tokens, const uw_rope *r, const uw_kv4_rows *q, int32_t q_heads,
                                        const uw_kv4_rows *q_out, const uw_kv4_rows *k, const uw_kv4_rows *v,
                                        const uw_kv4_rows *k_out, void *ws, size_t ws_bytes, void *stream) {
    if (!r)
        return UW_ERR_INVALID_ARG;
    return run_append(c, start, len, n_tokens, q, q_heads, q_out, k, v, r->cos_dev, r->sin_dev, r->rope_len,
                      r->rot_dim, r->interleaved, r, k_out, ws, ws_bytes, stream);
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
    const int chunk = rounds_of(n_tokens, rounds, 8);
    const int64_t units = n_tokens * ((rounds + chunk - 1) / chunk);
    if (units > int64_t(8) * 0x7fffffff)
        return UW_ERR_UNSUPPORTED;
    const dim3 grid(unsigned((units + 7) / 8));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto run = [&](auto kernel) { return launch_overlapped(kernel, grid, dim3(256), 0, st, view, ko, vo, chunk); };
    const cudaError_t e = c->head_dim == 128 ? (chunk > 1 ? run(kv4_read_kernel<128, 8>) : run(kv4_read_kernel<128, 1>))
                                             : (chunk > 1 ? run(kv4_read_kernel<64, 8>) : run(kv4_read_kernel<64, 1>));
    return e == cudaSuccess ? UW_OK : UW_ERR_CUDA;
}
