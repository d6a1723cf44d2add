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

// How a warp takes the heads of one token: `lanes` lanes for a head, eight pairs each, both sides; `per` heads at
// once, `rounds` times, `units` warps a token; what is not rotated has `tail` 16-byte steps a head.
struct RopePlan {
    int32_t half, lanes, per, rounds, units, tail;
    RopePlan() = default;
    RopePlan(int64_t tokens, int heads, int rot, int head_dim, int64_t warps) {
        half = rot / 2;
        lanes = rot / 16;
        per = 32 / lanes;
        tail = (head_dim - rot) / 8;
        const int all = (heads + per - 1) / per;
        // `warps` (two a scheduler) come first, longer ones after that
        rounds = 1;
        while (2 * rounds <= 16 && rounds < all && tokens * ((all + 2 * rounds - 1) / (2 * rounds)) >= warps)
            rounds *= 2;
        units = (all + rounds - 1) / rounds;
        rounds = (all + units - 1) / units;
    }
};

constexpr int kRopeAhead = 2;  // heads a lane has on their way

// Heads from `first` on (below `heads`) of a warp's token rotated: src(j) and dst(j) are where head j lies.  find()
// looks the token up, while the first heads are on their way; false: nothing is to be touched.  A lane reads
// what it writes, so dst may be src.
template <bool kInterleaved, class Src, class Dst, class Find>
__device__ __forceinline__ void rope_heads(const RopePlan &p, const Axes &axes, const float *cos, const float *sin,
                                           uint64_t zero, int first, int heads, Src src, Dst dst, Find find) {
    const int lane = threadIdx.x & 31;
    const int mine = lane / p.lanes, pc = lane - mine * p.lanes;
    const bool busy = mine < p.per;
    const int at0 = kInterleaved ? 16 * pc : 8 * pc, at1 = kInterleaved ? at0 + 8 : p.half + at0;
    uint4 x[kRopeAhead][2];
    auto fetch = [&](int n0) {
#pragma unroll
        for (int n = 0; n < kRopeAhead; n++) {
            const int j = first + (n0 + n) * p.per + mine;
            const bool in = busy && n0 + n < p.rounds && j < heads;
            const uint16_t *const at = src(in ? j : first);
            x[n][0] = in ? *reinterpret_cast<const uint4 *>(at + at0) : make_uint4(0, 0, 0, 0);
            x[n][1] = in ? *reinterpret_cast<const uint4 *>(at + at1) : make_uint4(0, 0, 0, 0);
        }
    };
    fetch(0);
    AxesAt turn;
    if (!find(turn))
        return;
    Rotation r[2];
    r[0].on = r[1].on = true;
    r[0].interleaved = r[1].interleaved = kInterleaved;
    if (busy) {
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const float4 cs = turn.four(axes, cos, p.half, 8 * pc + 4 * k);
            const float4 sn = turn.four(axes, sin, p.half, 8 * pc + 4 * k);
            if (kInterleaved) {
                r[k].of_pairs(cs, sn);
            } else {
                r[0].of_side(cs, sn, k, false);
                r[1].of_side(cs, sn, k, true);
            }
        }
    }
    for (int n0 = 0; n0 < p.rounds;) {
#pragma unroll
        for (int n = 0; n < kRopeAhead; n++) {
            const int j = first + (n0 + n) * p.per + mine;
            uint32_t a[4] = {x[n][0].x, x[n][0].y, x[n][0].z, x[n][0].w};
            uint32_t b[4] = {x[n][1].x, x[n][1].y, x[n][1].z, x[n][1].w};
            rotate(r[0], zero, a, x[n][1]);
            rotate(r[1], zero, b, x[n][0]);
            if (busy && n0 + n < p.rounds && j < heads) {
                uint16_t *const at = dst(j);
                *reinterpret_cast<uint4 *>(at + at0) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4 *>(at + at1) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        }
        n0 += kRopeAhead;
        if (n0 < p.rounds)
            fetch(n0);
    }
    if (!p.tail)
        return;
    const int last = min(first + p.rounds * p.per, heads);
    for (int i = lane; i < (last - first) * p.tail; i += 32) {
        const int j = first + i / p.tail, at = 2 * p.half + 8 * (i % p.tail);
        const uint16_t *const from = src(j) + at;
        uint16_t *const to = dst(j) + at;
        if (from != to)
            *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
    }
}

// rope.cu: the caller's axes, checked, as the kernels take them.
uw_status rope_axes_map(const uw_rope &r, int64_t n_tokens, Axes *a);

}  // namespace uw
