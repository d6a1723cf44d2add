// Attention over the 4-bit paged cache for sequences with few rows (new
// tokens x query heads of a kv head): single tokens, drafted tokens.
//
// Every cached vector is read once for all rows that share it, D / 2 + 4 bytes,
// so memory is the floor; what bounds the kernel is what a warp does with 32 keys
// of 128 (4352 bytes): 555 instructions, 160 of them the logic that takes the
// codes apart and 64 the subtractions of their middle, at 0.62 instructions a
// cycle, which 0.9 of a copy's rate is not far from.  A CTA of eight warps takes an equal share of all key
// tiles (kv4_attn.cuh), and each of its warps an equal share of that, which it
// works through by itself: a ring of tiles in flight (cp.async) runs on from
// item to item, an item that lies in one warp's share is written out by that
// warp, and only the items that the cuts between warps and CTAs go through
// are joined at the end, first in the CTA, then through the workspace.
//
// The products run on mma.sync.m16n8k16 with keys (and dimensions) on the
// 16-row side and 8 rows of queries on the other, so that 8 rows cost no
// more than one and the codes are the A operand straight from shared memory
// registers; tcgen05 would pad the rows to 64 or 128 and needs its operands
// written out as BF16.
//   S^T = K Q^T   a code is a BF16 as it stands (see Codes: one logic operation
//                 for two), and the scale and offset of a key are applied to
//                 the fp32 product: q.k = s sum q c + lo sum q.  Exact but for
//                 fp32 sums: no rounded K.
//   O^T = V^T P^T the codes of two keys come side by side out of a transposing
//                 matrix load.  A code becomes c - 8 (one subtraction more: without
//                 it the sum over many keys would lose digits to the offset, and
//                 subtracting 8 sum p s from the products in fp32 left 2^-24 of a
//                 large p where a value is exactly zero), the scale goes into the
//                 probability, p s, and the middle of the range into a sum of its
//                 own: o = sum (p s)(c - 8) + sum p (lo + 8 s).  p s is taken
//                 as the sum of two BF16, a rounding and its rest, so that the
//                 result is exact to about 2^-16 before its own rounding.  Up
//                 to four rows leave half of the products' columns empty: the
//                 rests go there (the same rows again) and cost nothing; more
//                 rows take a second product.
// The running maximum of the softmax is only raised when a score passes it by
// 2^24 (BF16 and fp32 hold that without loss), so that a tile costs a vote
// in place of shuffles.
//
// Measured, 32 query and 8 kv heads of 128:
//   one token, 131071 keys       39.3 us (3.6 TB/s)
//   one token, 1048576 keys      203 us (5.6 TB/s, of 6.8 for a copy); keys more cost at 6.1 TB/s
//   64 tokens, 40 to 8192 keys   37 us (3.0 TB/s)
//   one token, 257 keys          8.2 us
// A call's first 6 us go to finding the shares and the first loads, its last
// 6 to the joins, whose steps wait for one another's loads.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kernels.h"
#include "kv4_attn.cuh"
#include "kv4_codes.cuh"
#include "tc.cuh"

namespace uw {

namespace {

constexpr int kWarps = 8;
constexpr int kTile = 32;            // keys of a unit
constexpr float kRaise = 24.f;       // log2 headroom of a probability
// What an item costs a warp beyond its tiles (queries, output), in tiles: 64
// tokens of 40 to 8192 keys 45.8 us with none, 40.5 with 1, 38.4 with 2, 37.8 with 3, 38.0 with 4.
constexpr int kItemCost = 3;
// Items up to this many tiles are not cut between CTAs while shares are short:
// one token of 257 keys 11.2 us if they are, 8.6 if not.
constexpr uint32_t kWholeTiles = 32;
// Sequences of more than eight rows are taken sixteen at a time (each key
// unpacked once for all, but one CTA an SM) only if there are more units (32 keys
// x 8 rows) than this: 16 x 4 new tokens, 4096 keys 41 us against 46 by eights,
// 1 x 4 new tokens, 8192 keys 18.9 us against 17.7, 7 x 5 drafted tokens 18.1 against 15.1.
constexpr int64_t kNarrow = 32768;

template <int D>
constexpr int kStageBytes = kTile * (D + 8);
template <int D>
constexpr int kStages = D == 128 ? 3 : 5;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// A product's 16 keys: row 8 h + i of product mt stands for key 4 i + 2 mt + h
// of the tile, so that a lane's four keys (i = g) and their scales and offsets
// lie side by side.  Rows of codes lie in 128-byte lines, several to a line,
// and the 16-byte chunks of a line are exchanged by turn(row / 4): the rows
// 4 i + .. of eight (or, for the wider loads of K, of a phase's) lanes are then
// on different banks.
template <int D>
__device__ __forceinline__ uint32_t turn(uint32_t i) {
    return (D == 128 ? (i & 1) << 2 | i >> 1 : i << 1 | i >> 2) & 7;
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane (g, t) gets rows 2t
// and 2t + 1 of column g of each; lane 8 i + r gives the address of row r of matrix i.
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

template <int D, int NT>
struct Warp {
    // D/16 pairs of dimensions of the output for 2 rows of each of NT row groups
    float o[D / 16][NT][4];
    float m[NT][2];
    uint64_t l[NT], z[NT];   // sums of p and of p (lo + 8 s), for the two rows
    uint32_t q[NT][D / 16][2];
    uint64_t qs[NT];         // sum of q
};

constexpr int kSegs = 8;  // segments a warp lists at once

// A part of an item that waits to be joined.
struct Part {
    const float *at;  // its floats; null: none
    uint64_t u0;
    int32_t rt, t0, tokens, head, tiles, of;
};

// NT groups of eight rows; kDup (NT = 1): up to four rows, which rows 4..7 repeat
// (one token, 131071 keys 40.6 us, with a second product for the rests 44.2).
template <int D, int NT, bool kDup>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 2 : 1) kv4_decode_kernel(const AttnParams p) {
    static_assert(!kDup || NT == 1, "rows repeated in one group");
    constexpr int RB = kDup ? 4 : 8 * NT;
    constexpr int ST = kStages<D>;
    constexpr int PF = RB * (D + 2);  // floats of a part
    using S = Sched<RB, kTile, kItemCost>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Row<kWarps * 32> row_of_units;
    __shared__ Seg all_segs[kWarps][kSegs];
    __shared__ Part parts[2 * kWarps], pend[2];
    __shared__ float row_m[RB], row_l[RB];
    __shared__ uint32_t arrived[2], from[2], to_part[2];
    grid_dep_launch();
    grid_dep_wait();
    const Kv4View &v = p.v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    unsigned char *const ring = smem + warp * ST * kStageBytes<D>;
    const uint32_t ring_at = smem_addr(ring);
    if (lane < 2)
        parts[2 * warp + lane].at = nullptr;
    if (threadIdx.x < 2)
        pend[threadIdx.x].at = nullptr;

    // this CTA's share [cut 0, cut 1) of the units, and this warp's of that
    const uint64_t total = build_row<S, kWarps * 32, false>(p, row_of_units);
    const uint32_t workers = uint32_t(min(total, uint64_t(gridDim.x)));
    if (blockIdx.x >= workers)
        return;
    uint64_t cut[2] = {mul_div(total, blockIdx.x, workers), mul_div(total, blockIdx.x + 1, workers)};
    // While a share is about a tile for each warp, an item of a few tiles a
    // warp is taken whole: a cut through it would cost a round trip through
    // the workspace.
    const bool snap = total <= uint64_t(kWarps + kItemCost) * gridDim.x;
    uint64_t u = cut[0], u_end = cut[1];
    Item it{};
    bool found = false;  // `it` holds unit u
#pragma unroll 1
    for (int k = snap ? 0 : 2; k < 3; k++) {
        const uint64_t end = it.u0 + it.n;
        if (k == 1) {
            if (cut[1] == total || cut[1] == end)
                continue;
            if (cut[1] < end) {  // in the same item
                cut[1] = it.tiles <= kWholeTiles ? it.u0 : cut[1];
                continue;
            }
        }
        if (k == 2) {
            if (cut[0] == cut[1])
                return;
            u = cut[0] + (cut[1] - cut[0]) * warp / kWarps;
            u_end = cut[0] + (cut[1] - cut[0]) * (warp + 1) / kWarps;
            if (u == u_end || (found && u >= it.u0 && u < end))
                break;
        }
        const Item at = locate<S>(p, row_of_units, k == 1 ? cut[1] : u);
        if (k < 2 && at.tiles <= kWholeTiles)
            cut[k] = at.u0;
        if (k != 1) {
            it = at;
            found = true;
        }
    }
    Seg *const segs = all_segs[warp];
    const int64_t block = int64_t(D + 8) << v.page_log2;
    const uint32_t page_bytes = uint32_t(block) * v.heads;  // (at most 65536 heads of 34816 bytes)
    const int mask = (1 << v.page_log2) - 1;
    const uint32_t v_off = (D / 2) << v.page_log2;

    // The warp's next tile to copy runs ahead of the products through all listed
    // segments.  Lanes 0..15 copy its keys 0..15, the others the rest (which may
    // lie in another page of 16): nx_key is the lane's first, nx_page its page.  A
    // tile's keys are always copied in full, they are there in the page; what
    // no row sees is left out of the sums.
    int n_segs = 0, nx_seg = 0, nx_tiles = 0, nx_key = 0, nx_last = 0, nx_page = 0;
    const uint8_t *nx_base = nullptr;
    const int32_t *nx_table = nullptr;
    bool bad = false;
    auto next_seg = [&]() {
        while (nx_seg < n_segs && segs[nx_seg].tiles == 0)
            nx_seg++;
        if (nx_seg == n_segs)
            return;
        const Seg &sg = segs[nx_seg++];
        nx_tiles = sg.tiles;
        nx_key = sg.first * kTile + (lane & 16);
        nx_last = sg.len - 1;
        nx_base = v.pages + (sg.head * block + (lane & 15) * 16);
        nx_table = v.table + int64_t(sg.s) * v.table_stride;
        nx_page = __ldg(nx_table + (min(max(nx_key, sg.lo), nx_last) >> v.page_log2));
    };
    constexpr int RC = D / 32;  // 16-byte chunks of a row
    const uint32_t first_row = (lane & 16) + (lane & 15) / RC;
    const uint32_t to0 = ((first_row * RC + lane % RC) ^ turn<D>(first_row >> 2)) * 16;
    // scales and offsets: from the lane's first codes
    const uint32_t par_off = kv4_params<D>(v.page_log2, 0, (lane >> 2) & 1) - (lane & 12) * 16;
    const uint32_t par_to = kTile * D + ((lane & 4) ? kTile * 4 : 0) + ((lane & 16) ? 64 : 0) + (lane & 3) * 16;
    auto issue = [&](int stage) {
        if (nx_tiles > 0) {
            const uint32_t dst = ring_at + stage * kStageBytes<D>;
            const bool ok = uint32_t(nx_page) < uint64_t(v.n_pages);  // (looked at here, not where it is loaded)
            bad = bad || !ok;
            const uint32_t slot = nx_key & mask, bytes = ok ? 16 : 0;
            const uint8_t *const page = nx_base + uint64_t(ok ? nx_page : 0) * page_bytes;
            const uint8_t *const src = page + slot * (D / 2);
#pragma unroll
            for (int j = 0; j < RC; j++) {
                // rows first_row + 16 / RC j; what that does to their turn
                constexpr uint32_t kStep = D == 128 ? 1 : 2;
                const uint32_t to = dst + (to0 ^ (turn<D>(kStep * j) * 16)) + j * 256;
                cp_async16_zfill(to, src + j * 256, bytes);
                cp_async16_zfill(to + kTile * (D / 2), src + (v_off + j * 256), bytes);
            }
            if ((lane & 8) == 0)
                cp_async16_zfill(dst + par_to, page + (slot * 4 + par_off), bytes);
            if (--nx_tiles == 0) {
                next_seg();
            } else {
                nx_key += kTile;
                nx_page = __ldg(nx_table + (min(nx_key, nx_last) >> v.page_log2));
            }
        }
        cp_async_commit();
    };

    const Codes codes;
    const float c1_up = p.c1 * kQDown;
    int stage = 0;  // the ring's next stage to use
    while (u < u_end) {
        u = list_segments<S, kSegs>(p, it, u, u_end, segs, &n_segs);
        nx_seg = 0;
        next_seg();
        int fill = stage, to_fill = ST;
        for (int sgi = 0; sgi < n_segs; sgi++) {
            const Seg &sg = segs[sgi];
            const int n_mine = sg.tiles;
            const int r0 = sg.rt * RB, rows = sg.tokens * p.group;
            const int all_lo = sg.all_lo, all_hi = sg.all_hi;
            const Seq sq{sg.t0, sg.tokens, sg.len};

            Warp<D, NT> w;
            // Queries: lane (g, t) holds row g of each group, dimensions D/4 t .. + D/4 - 1,
            // paired as the codes of a word come out of it: (0,4) (1,5) (2,6) (3,7).
            uint4 xq[NT][D / 32];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const int rr = nt * 8 + (kDup ? g & 3 : g);
#pragma unroll
                for (int k = 0; k < D / 32; k++)
                    xq[nt][k] = make_uint4(0, 0, 0, 0);
                if (rr < rows - r0 && n_mine > 0) {
                    const int i = p.by_group.of(r0 + rr);
                    const int64_t tok = sg.t0 + i, head = sg.head * p.group + (r0 + rr - i * p.group);
                    const uint16_t *at = p.q.p + tok * p.q.ts + head * p.q.hs + (D / 4) * t;
                    const uint4 *src = reinterpret_cast<const uint4 *>(at);
#pragma unroll
                    for (int k = 0; k < D / 32; k++)
                        xq[nt][k] = src[k];
                }
            }
            // the ring's fill, while the first queries are on their way
#pragma unroll 1
            for (; to_fill > 0; to_fill--) {
                issue(fill);
                fill = fill + 1 == ST ? 0 : fill + 1;
            }
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const uint4(&x)[D / 32] = xq[nt];
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < D / 32; k++) {
                    w.q[nt][2 * k][0] = mul2_bf16(__byte_perm(x[k].x, x[k].z, 0x5410), kQUpLow);
                    w.q[nt][2 * k][1] = mul2_bf16(__byte_perm(x[k].x, x[k].z, 0x7632), kQUpHigh);
                    w.q[nt][2 * k + 1][0] = mul2_bf16(__byte_perm(x[k].y, x[k].w, 0x5410), kQUpLow);
                    w.q[nt][2 * k + 1][1] = mul2_bf16(__byte_perm(x[k].y, x[k].w, 0x7632), kQUpHigh);
                    const uint32_t a[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        sum += bf16_lo(a[i]) + bf16_hi(a[i]);
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                w.qs[nt] = pair2(__shfl_sync(0xffffffffu, sum, 8 * t), __shfl_sync(0xffffffffu, sum, 8 * t + 4));
                w.m[nt][0] = w.m[nt][1] = -INFINITY;
                w.l[nt] = w.z[nt] = 0;
#pragma unroll
                for (int i = 0; i < D / 16; i++)
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        w.o[i][nt][k] = 0.f;
            }

            for (int i = 0; i < n_mine; i++) {
                asm volatile("cp.async.wait_group %0;" :: "n"(ST - 1) : "memory");
                __syncwarp();
                const unsigned char *const st = ring + stage * kStageBytes<D>;
                const uint32_t st_at = ring_at + stage * kStageBytes<D>;
                stage = stage + 1 == ST ? 0 : stage + 1;
                const int key0 = (sg.first + i) * kTile;

                // scores
                float sc[2][NT][4];
#pragma unroll
                for (int mt = 0; mt < 2; mt++)
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            sc[mt][nt][k] = 0.f;
                uint32_t a[4][D / 32];  // [key 4 g + j][words]
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    // row 4 g + j, bytes D / 8 t ..
                    const uint32_t s0 = D == 128 ? g * 16 + (t ^ turn<D>(g)) : g * 8 + ((t >> 1) ^ turn<D>(g));
                    const unsigned char *at = st + ((s0 * 16) ^ (D == 128 ? (j & 1) * 64 : j * 32)) +
                                              (D == 128 ? (j >> 1) * 128 : (t & 1) * 8);
                    if constexpr (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(at);
                        a[j][0] = x.x, a[j][1] = x.y, a[j][2] = x.z, a[j][3] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(at);
                        a[j][0] = x.x, a[j][1] = x.y;
                    }
                }
#pragma unroll
                for (int k = 0; k < D / 32; k++)
#pragma unroll
                    for (int j = 0; j < 2; j++)
#pragma unroll
                        for (int mt = 0; mt < 2; mt++) {
                            const uint32_t x = j ? a[2 * mt][k] >> 8 : a[2 * mt][k];
                            const uint32_t y = j ? a[2 * mt + 1][k] >> 8 : a[2 * mt + 1][k];
                            const uint32_t a0 = codes.low(x), a1 = codes.low(y), a2 = codes.high(x), a3 = codes.high(y);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
                                mma16816(sc[mt][nt], a0, a1, a2, a3, w.q[nt][2 * k + j][0], w.q[nt][2 * k + j][1]);
                        }
                // sc[mt][nt][2 h + k]: key 4 g + 2 mt + h, row 8 nt + 2 t + k.
                // In log2 units and less the maximum: y - m = acc * a + (c * qs - m).
                const uint4 kp = *reinterpret_cast<const uint4 *>(st + kTile * D + g * 16);
                const uint4 vp = *reinterpret_cast<const uint4 *>(st + kTile * (D + 4) + g * 16);
                const uint32_t kpar[4] = {kp.x, kp.y, kp.z, kp.w}, vpar[4] = {vp.x, vp.y, vp.z, vp.w};
                const bool open = key0 < all_lo || all_hi - key0 < kTile;  // (key0 + kTile may be 2^31)
                uint64_t y[4][NT];
                auto scores = [&]() {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float a = bf16_lo(kpar[j]) * c1_up, c = bf16_hi(kpar[j]) * p.c1;
                        const uint64_t aa = pair2(a, a), cc = pair2(c, c);
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
                            y[j][nt] = fma2(pair2(sc[j >> 1][nt][2 * (j & 1)], sc[j >> 1][nt][2 * (j & 1) + 1]), aa,
                                            fma2(cc, w.qs[nt], pair2(-w.m[nt][0], -w.m[nt][1])));
                    }
                    if (open) {
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) {
                            bool in[4][2];
#pragma unroll
                            for (int k = 0; k < 2; k++) {
                                const int row = 8 * nt + (kDup ? (2 * t + k) & 3 : 2 * t + k);
                                const int tok = p.by_group.of(r0 + min(row, rows - r0 - 1));
                                const KeyRange kr = visible(p, sq, tok, tok);
#pragma unroll
                                for (int j = 0; j < 4; j++) {
                                    const int key = key0 + 4 * g + j;
                                    in[j][k] = key >= kr.lo && key < min(kr.hi, sq.len);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                const float2 f = unpair(y[j][nt]);
                                y[j][nt] = pair2(in[j][0] ? f.x : -INFINITY, in[j][1] ? f.y : -INFINITY);
                            }
                        }
                    }
                };
                scores();
                // raise the maximum where a score passes it by far
                float top[NT][2];
                auto highest = [&](int nt) {
                    const float2 a = unpair(y[0][nt]), b = unpair(y[1][nt]), c = unpair(y[2][nt]), d = unpair(y[3][nt]);
                    top[nt][0] = fmaxf(fmaxf(a.x, b.x), fmaxf(c.x, d.x));
                    top[nt][1] = fmaxf(fmaxf(a.y, b.y), fmaxf(c.y, d.y));
                };
                bool raise = false;
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    highest(nt);
                    raise = raise || fmaxf(top[nt][0], top[nt][1]) > kRaise;
                }
                if (__any_sync(0xffffffffu, raise)) {
                    // With no maximum yet the scores are taken again, less nothing.
                    bool none = false;
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int k = 0; k < 2; k++)
                            none = none || w.m[nt][k] == -INFINITY;
                    const bool fresh = __any_sync(0xffffffffu, none);
                    float old[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            old[nt][k] = w.m[nt][k];
                            if (fresh)
                                w.m[nt][k] = 0.f;
                        }
                    if (fresh) {
                        scores();
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
                            highest(nt);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        float f[2];
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            float x = top[nt][k];
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                            const float m2 = fmaxf(old[nt][k], x + w.m[nt][k]);
                            f[k] = m2 == -INFINITY ? 1.f : exp2_fast(old[nt][k] - m2);
                            w.m[nt][k] = m2;
#pragma unroll
                            for (int d = 0; d < D / 16; d++) {
                                w.o[d][nt][k] *= f[k];
                                w.o[d][nt][2 + k] *= f[k];
                            }
                        }
                        w.l[nt] = mul2(w.l[nt], pair2(f[0], f[1]));
                        w.z[nt] = mul2(w.z[nt], pair2(f[0], f[1]));
                    }
                    scores();
                }
                // probabilities, as the B operand of the product with V: p s in two BF16
                uint32_t hi[2][NT][2], lo[2][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float s = bf16_lo(vpar[j]) * kPUp, mid = fmaf(8.f / kPUp, s, bf16_hi(vpar[j]));
                        const float2 f = unpair(y[j][nt]);
                        const uint64_t pr = pair2(exp2_fast(f.x), exp2_fast(f.y));
                        uint64_t ps = mul2(pr, pair2(s, s));
                        w.l[nt] = add2(w.l[nt], pr);
                        if (open) {  // a masked key's scale may be anything
                            const float2 a = unpair(ps), b = unpair(mul2(pr, pair2(mid, mid)));
                            const bool in0 = f.x != -INFINITY, in1 = f.y != -INFINITY;
                            ps = pair2(in0 ? a.x : 0.f, in1 ? a.y : 0.f);
                            w.z[nt] = add2(w.z[nt], pair2(in0 ? b.x : 0.f, in1 ? b.y : 0.f));
                        } else {
                            w.z[nt] = fma2(pr, pair2(mid, mid), w.z[nt]);
                        }
                        const float2 a = unpair(ps);
                        const uint32_t h = bf16_pack(a.x, a.y);
                        const float2 rest = unpair(add2(ps, pair2(-bf16_lo(h), -bf16_hi(h))));
                        const uint32_t r = bf16_pack(rest.x, rest.y);
                        if constexpr (kDup) {
                            hi[j >> 1][nt][j & 1] = transpose8x8(t < 2 ? h : r);
                        } else {
                            hi[j >> 1][nt][j & 1] = transpose8x8(h);
                            lo[j >> 1][nt][j & 1] = transpose8x8(r);
                        }
                    }
                // output
#pragma unroll
                for (int mt = 0; mt < 2; mt++)
#pragma unroll
                    for (int c = 0; c < D / 64; c++) {
                        // x[2 e + h]: rows 8 h + 2t, + 1, the four codes 4 g .. of chunk 2 c + e
                        uint32_t x[4];
                        const uint32_t i = lane & 7, h = (lane >> 3) & 1, e0 = lane >> 4;
                        const uint32_t s0 = i * (D / 8) + ((h * (D / 32) + e0) ^ turn<D>(i));
                        ldmatrix_t(x, st_at + kTile * (D / 2) + ((s0 * 16) ^ (D == 128 ? c * 32 : mt * 64)) +
                                          (D == 128 ? mt * 128 : 0));
#pragma unroll
                        for (int e = 0; e < 2; e++)
#pragma unroll
                            for (int j = 0; j < 2; j++) {
                                const uint32_t y = x[2 * e] >> 8 * j, z = x[2 * e + 1] >> 8 * j;
                                const uint32_t a0 = codes.low_mid(y), a1 = codes.high_mid(y);
                                const uint32_t a2 = codes.low_mid(z), a3 = codes.high_mid(z);
#pragma unroll
                                for (int nt = 0; nt < NT; nt++) {
                                    float(&o)[4] = w.o[4 * c + 2 * e + j][nt];
                                    mma16816(o, a0, a1, a2, a3, hi[mt][nt][0], hi[mt][nt][1]);
                                    if constexpr (!kDup)
                                        mma16816(o, a0, a1, a2, a3, lo[mt][nt][0], lo[mt][nt][1]);
                                }
                            }
                    }
                __syncwarp();
                issue(fill);  // a tile for a tile
                fill = fill + 1 == ST ? 0 : fill + 1;
            }
            // A whole item is written out; a part of one goes to the workspace, or
            // (the warp's last) to its ring.
            const bool whole = sg.tiles == sg.of;
            const bool last = u == u_end && sgi == n_segs - 1;
            float *part = nullptr;
            if (!whole) {
                if (last) {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    __syncwarp();
                }
                part = last ? reinterpret_cast<float *>(ring)
                            : p.parts + (2 * uint64_t(gridDim.x) + blockIdx.x * kWarps + warp) * PF;
                if (lane == 0)
                    parts[2 * warp + last] = Part{part, sg.u0, sg.rt, sg.t0, sg.tokens, sg.head, sg.tiles, sg.of};
            }
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const float2 l2 = unpair(w.l[nt]), z2 = unpair(w.z[nt]);
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    float l = k ? l2.y : l2.x, z = k ? z2.y : z2.x;
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        l += __shfl_xor_sync(0xffffffffu, l, o);
                        z += __shfl_xor_sync(0xffffffffu, z, o);
                    }
                    float o[D / 8];  // o[4 c + i]: dimension 32 c + 4 g + i of row 8 nt + 2 t + k
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        o[2 * i] = w.o[i][nt][k] * kPDownLow;
                        o[2 * i + 1] = w.o[i][nt][2 + k] * kPDownHigh;
                    }
                    if constexpr (kDup) {  // the rests' products are in the columns four on
#pragma unroll
                        for (int i = 0; i < D / 8; i++)
                            o[i] += __shfl_xor_sync(0xffffffffu, o[i], 2);
                    }
#pragma unroll
                    for (int i = 0; i < D / 8; i++)
                        o[i] += z;
                    const int row = 8 * nt + 2 * t + k;
                    if ((!kDup || t < 2) && r0 + row < rows) {
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < D / 32; i++)
                                store_row<D>(p, sg.t0, sg.head, r0 + row, 8 * i + g,
                                             make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]),
                                             w.m[nt][k], l);
                        } else {
                            float4 *const dst = reinterpret_cast<float4 *>(part) + row * (D / 4) + g;
#pragma unroll
                            for (int i = 0; i < D / 32; i++)
                                dst[8 * i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            if (g == 0) {
                                part[RB * D + row] = w.m[nt][k];
                                part[RB * D + RB + row] = l;
                            }
                        }
                    }
                }
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (bad)
        atomicOr(v.status, kStatusBadCache);
    __syncthreads();

    // Items that the cuts between the warps go through: consecutive parts of
    // one item are joined, in their order, and written out or, if the CTA does
    // not have all of the item, left in the workspace.  Lane i of every warp looks
    // at part i: a group begins where the item is not the part's before.
    {
        const bool has = lane < 2 * kWarps && parts[lane & (2 * kWarps - 1)].at;
        const uint64_t id = has ? parts[lane].u0 : 0;
        const uint32_t some = __ballot_sync(0xffffffffu, has);
        const uint32_t under = some & ((1u << lane) - 1u);
        const uint64_t id_before = __shfl_sync(0xffffffffu, id, under ? 31 - __clz(under) : 0);
        uint32_t heads = __ballot_sync(0xffffffffu, has && (under == 0 || id_before != id));
        const int n = __popc(heads) * (RB * D / 4);
        int at_group = 0;
        for (int idx = threadIdx.x; idx < n; idx += kWarps * 32) {
            for (; at_group < idx / (RB * D / 4); at_group++)
                heads &= heads - 1;
            const int a = __ffs(heads) - 1, x = idx % (RB * D / 4), row = x / (D / 4);
            const uint32_t later = heads & (heads - 1);
            const int b = later ? __ffs(later) - 1 : 2 * kWarps;
            const Part &head = parts[a];
            const int r0 = head.rt * RB;
            if (row >= head.tokens * p.group - r0)
                continue;
            // every part's place in the loops is known, so that their loads go out together
            const uint32_t in = some & ((2u << (b - 1)) - (1u << a));
            float w[2 * kWarps], m = -INFINITY, l = 0.f;
            int tiles = 0;
#pragma unroll
            for (int k = 0; k < 2 * kWarps; k++) {
                const Part &part = parts[in >> k & 1 ? k : a];
                w[k] = in >> k & 1 ? part.at[RB * D + row] : -INFINITY;
                tiles += in >> k & 1 ? part.tiles : 0;
                m = fmaxf(m, w[k]);
            }
            const float m0 = m == -INFINITY ? 0.f : m;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 2 * kWarps; k++)
                if (in >> k & 1) {
                    const float *q = parts[k].at;
                    join_scaled(l, acc, exp2_fast(w[k] - m0), q[RB * D + RB + row],
                                reinterpret_cast<const float4 *>(q)[x]);
                }
            const int c = x % (D / 4);
            if (tiles == head.of) {
                store_row<D>(p, head.t0, head.head, r0 + row, c, acc, m, l);
            } else {
                const int first = cut[0] > head.u0 ? 0 : 1;  // ends an item, or begins one
                float *const part = p.parts + (2 * uint64_t(blockIdx.x) + first) * PF;
                reinterpret_cast<float4 *>(part)[x] = acc;
                if (c == 0) {
                    part[RB * D + row] = m;
                    part[RB * D + RB + row] = l;
                }
                if (x == 0) {
                    pend[first] = head;
                    pend[first].at = part;
                }
            }
        }
    }
    __syncthreads();
    if (pend[0].at == nullptr && pend[1].at == nullptr)
        return;
    __threadfence();
    __syncthreads();

    // Items that go on in other CTAs: whoever arrives last joins the parts.
    if (threadIdx.x < 2 && pend[threadIdx.x].at) {
        const Part &sg = pend[threadIdx.x];
        const uint32_t f = share_of(sg.u0, total, workers), e = share_of(sg.u0 + sg.of - 1, total, workers);
        const bool last = atomicAdd(p.counters + f, 1u) == e - f;
        if (last)
            p.counters[f] = 0;  // ready for the next call
        arrived[threadIdx.x] = last;
        from[threadIdx.x] = f;
        to_part[threadIdx.x] = e;
    }
    __syncthreads();
    for (int k = 0; k < 2; k++) {
        if (pend[k].at == nullptr || !arrived[k])
            continue;
        __threadfence();
        // Every part's maximum and sum give its weight; the outputs are on their
        // way meanwhile: thread x takes float4 x of every second (or fourth, ...)
        // part, and the threads of one float4 are added in their order.
        const Part &sg = pend[k];
        const uint32_t f = from[k];
        const int n = int(to_part[k] - f) + 1;
        const int r0 = sg.rt * RB, real = min(sg.tokens * p.group - r0, RB);
        const int f4 = real * (D / 4);
        auto part_of = [&](int i) { return p.parts + (2 * uint64_t(f + i) + (i == 0 ? 1 : 0)) * PF; };
        float *const wt = reinterpret_cast<float *>(smem);             // [n][RB] weights
        float *const sums = wt + n * RB;                               // [n][RB] sums, then outputs
        for (int i = threadIdx.x; i < n * RB; i += kWarps * 32) {
            const bool in = i % RB < real;
            wt[i] = in ? __ldcg(part_of(i / RB) + RB * D + i % RB) : -INFINITY;
            sums[i] = in ? __ldcg(part_of(i / RB) + RB * D + RB + i % RB) : 0.f;
        }
        constexpr int F4 = RB * (D / 4);
        constexpr int kSplit = F4 < kWarps * 32 ? kWarps * 32 / F4 : 1, kTurns = F4 * kSplit / (kWarps * 32);
        constexpr int kHeld = 16;
        float4 *const outs = reinterpret_cast<float4 *>(smem + (2 * n * RB * 4 + 15) / 16 * 16);
        const int s0 = threadIdx.x / F4 % kSplit;
#pragma unroll
        for (int turn = 0; turn < kTurns; turn++) {
            const int x = threadIdx.x % F4 + turn * (kWarps * 32), row = x / (D / 4);
            float4 held[kHeld];
#pragma unroll
            for (int h = 0; h < kHeld; h++) {
                const int i = s0 + h * kSplit;
                held[h] = x < f4 && i < n ? __ldcg(reinterpret_cast<const float4 *>(part_of(i)) + x)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (turn == 0) {
                __syncthreads();
                for (int row = warp; row < real; row += kWarps) {  // a warp a row, a lane a part
                    float m = -INFINITY, l = 0.f;
                    for (int i = lane; i < n; i += 32)
                        m = fmaxf(m, wt[i * RB + row]);
#pragma unroll
                    for (int o = 16; o; o >>= 1)
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float m0 = m == -INFINITY ? 0.f : m;
                    for (int i = lane; i < n; i += 32) {
                        const float w = exp2_fast(wt[i * RB + row] - m0);
                        wt[i * RB + row] = w;
                        l = fmaf(w, sums[i * RB + row], l);
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1)
                        l += __shfl_xor_sync(0xffffffffu, l, o);
                    if (lane == 0) {
                        row_m[row] = m;
                        row_l[row] = l;
                    }
                }
                __syncthreads();
            }
            if (x >= f4)
                continue;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            auto add = [&](int i, const float4 &o) {
                const float w = wt[i * RB + row];
                acc.x = fmaf(w, o.x, acc.x);
                acc.y = fmaf(w, o.y, acc.y);
                acc.z = fmaf(w, o.z, acc.z);
                acc.w = fmaf(w, o.w, acc.w);
            };
#pragma unroll
            for (int h = 0; h < kHeld; h++)
                if (s0 + h * kSplit < n)
                    add(s0 + h * kSplit, held[h]);
#pragma unroll 8
            for (int i = s0 + kHeld * kSplit; i < n; i += kSplit)
                add(i, __ldcg(reinterpret_cast<const float4 *>(part_of(i)) + x));
            outs[s0 * F4 + x] = acc;
        }
        __syncthreads();
        for (int x = threadIdx.x; x < f4; x += kWarps * 32) {
            const int row = x / (D / 4);
            float4 acc = outs[x];
#pragma unroll
            for (int s0 = 1; s0 < kSplit; s0++) {
                const float4 o = outs[s0 * F4 + x];
                acc.x += o.x;
                acc.y += o.y;
                acc.z += o.z;
                acc.w += o.w;
            }
            store_row<D>(p, sg.t0, sg.head, r0 + row, x % (D / 4), acc, row_m[row], row_l[row]);
        }
        __syncthreads();
    }
}

template <int D, int NT, bool kDup>
uw_status launch(const AttnParams &p, int ctas, cudaStream_t st) {
    static_assert(8 * NT * (D + 2) * 4 <= kStages<D> * kStageBytes<D>, "a part fits a ring");
    constexpr size_t smem = size_t(kWarps) * kStages<D> * kStageBytes<D>;
    if (!ensure_smem(kv4_decode_kernel<D, NT, kDup>, smem))
        return UW_ERR_CUDA;
    return launch_overlapped(kv4_decode_kernel<D, NT, kDup>, dim3(unsigned(ctas)), dim3(kWarps * 32), smem, st, p) ==
                   cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}

}  // namespace

int kv4_decode_ctas() { return 2 * sm_count(); }

size_t kv4_decode_part_floats(int head_dim) { return (2 + kWarps) * size_t(kv4_decode_ctas()) * 16 * (head_dim + 2); }

uw_status launch_kv4_decode(const AttnParams &p, int head_dim, int64_t rows, int64_t max_units, cudaStream_t st) {
    const bool dup = rows > 0 && rows <= 4, wide = rows == 0 || (rows > 8 && (max_units == 0 || max_units > kNarrow));
    int64_t ctas = wide ? kv4_decode_ctas() / 2 : kv4_decode_ctas();
    if (max_units > 0)
        ctas = std::min(ctas, max_units);
    const int n = int(ctas);
    auto of = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        return wide  ? launch<D, 2, false>(p, n, st)
               : dup ? launch<D, 1, true>(p, n, st)
                     : launch<D, 1, false>(p, n, st);
    };
    return head_dim == 128 ? of(std::integral_constant<int, 128>()) : of(std::integral_constant<int, 64>());
}

}  // namespace uw
