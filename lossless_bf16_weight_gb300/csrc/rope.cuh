// Rotation of q and k by positions: on several axes (Axes), and what a lane
// multiplies with (Rotation).
#pragma once
#include "kv4.cuh"

namespace uw {

constexpr int kMaxAxes = 4, kMaxPairs = 128;

// Positions on n axes, an axis's `stride` from the next's, and the axis of each
// pair: two bits a pair, sixteen pairs a word.
struct Axes {
    const int32_t *pos;
    int64_t stride;
    int32_t n;
    uint32_t map[kMaxPairs / 16];
};

// One token's positions.
struct AxesAt {
    int32_t p[kMaxAxes] = {0, 0, 0, 0};
    // False if one is not a row of the tables.
    __device__ __forceinline__ bool find(const Axes &a, int64_t t, int64_t rope_len) {
        bool ok = true;
#pragma unroll
        for (int i = 0; i < kMaxAxes; i++)
            if (i < a.n)
                p[i] = __ldg(a.pos + i * a.stride + t);
#pragma unroll
        for (int i = 0; i < kMaxAxes; i++)
            ok = ok && (i >= a.n || (p[i] >= 0 && p[i] < rope_len));
        return ok;
    }
    __device__ __forceinline__ int32_t on(uint32_t axis) const {
        return axis == 0 ? p[0] : axis == 1 ? p[1] : axis == 2 ? p[2] : p[3];
    }
    // A table's values of pairs j .. j + 3 (j a multiple of four): one step where they turn
    // together.
    __device__ __forceinline__ float4 four(const Axes &a, const float *table, int pairs, int j) const {
        const uint32_t axis = (a.map[j >> 4] >> (2 * (j & 15))) & 0xffu;
        if (axis == (axis & 3u) * 0x55u)
            return __ldg(reinterpret_cast<const float4 *>(table + int64_t(on(axis & 3u)) * pairs + j));
        auto one = [&](int k) { return __ldg(table + int64_t(on((axis >> (2 * k)) & 3u)) * pairs + j + k); };
        return make_float4(one(0), one(1), one(2), one(3));
    }
};

// A lane's share of a token's rotation: its eight values are one side of
// eight pairs (half split: the other side lies rot / 2 values on or back), or four
// whole pairs (interleaved).
struct Rotation {
    uint64_t c[4], s[4];  // cosines and sines of two values each, the sines with the sign of the side
    bool on, interleaved;
    __device__ __forceinline__ void of_pairs(const float4 &cs, const float4 &sn) {
        c[0] = pair2(cs.x, cs.x), c[1] = pair2(cs.y, cs.y);
        c[2] = pair2(cs.z, cs.z), c[3] = pair2(cs.w, cs.w);
        s[0] = pair2(-sn.x, sn.x), s[1] = pair2(-sn.y, sn.y);
        s[2] = pair2(-sn.z, sn.z), s[3] = pair2(-sn.w, sn.w);
    }
    // Values 4 k .. 4 k + 3 of the first or second sides.
    __device__ __forceinline__ void of_side(const float4 &cs, const float4 &sn, int k, bool second) {
        const float sign = second ? 1.f : -1.f;
        c[2 * k] = pair2(cs.x, cs.y), c[2 * k + 1] = pair2(cs.z, cs.w);
        s[2 * k] = pair2(sign * sn.x, sign * sn.y), s[2 * k + 1] = pair2(sign * sn.z, sign * sn.w);
    }
};

// Rotated values of a lane, own c + other s: own ones in a, the other side's in
// b (half split).  Each product is rounded and then the sum: a product is a
// fused multiply-add to a -0 that comes with the call, as the assembler joins
// a plain product, and one with a -0 that it sees, with the sum.
__device__ __forceinline__ void rotate(const Rotation &r, uint64_t zero, uint32_t (&a)[4], const uint4 &other) {
    if (!r.on)
        return;
    const uint32_t b[4] = {other.x, other.y, other.z, other.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float u = bf16_lo(a[k]), w = bf16_hi(a[k]);
        const uint64_t o = r.interleaved ? pair2(w, u) : pair2(bf16_lo(b[k]), bf16_hi(b[k]));
        const float2 y = unpair(add2(fma2(pair2(u, w), r.c[k], zero), fma2(o, r.s[k], zero)));
        a[k] = bf16_pack(y.x, y.y);
    }
}

// rope.cu: the caller's axes, checked, as the kernels take them.
uw_status rope_axes_map(const uw_rope &r, int64_t n_tokens, Axes *a);

}  // namespace uw
