// Attention over the 4-bit paged cache for sequences with few rows (new
// tokens x query heads of a kv head): single tokens, drafted tokens.
//
// Bound by memory: every cached vector is read once for all rows that share
// it, D / 2 + 4 bytes.  A CTA of eight warps takes an equal share of all key
// tiles (kv4_attn.cuh); in it a warp takes every eighth tile of 32 keys and
// keeps a ring of tiles in flight by itself (cp.async, no CTA barrier), so
// that about 100 KB an SM are on their way.
//
// The products run on mma.sync.m16n8k16 with keys (and dimensions) on the
// 16-row side and 8 rows of queries on the other, so that 8 rows cost no
// more than one and the codes are the A operand straight from shared memory
// registers; tcgen05 would pad the rows to 64 or 128 and needs its operands
// written out as BF16.
//   S^T = K Q^T   a code c becomes BF16 16 + c by one logic operation (its
//                 bits are the upper mantissa bits of 16), and the scale and
//                 offset of a key are applied to the fp32 product:
//                 q.k = s (sum q (16 + c)) + (lo - 16 s) sum q.  Exact but for
//                 fp32 sums: no rounded K.
//   O^T = V^T P^T a code becomes c - 8 (one more subtraction: a sum over many
//                 keys would lose digits to the offset), the scale goes into
//                 the probability, p s, and the middle of the range into a sum
//                 of its own: o = sum (p s)(c - 8) + sum p (lo + 8 s).  p s is taken
//                 as the sum of two BF16 (a rounding and its rest), two
//                 products for each, which the tensor cores have room for: the
//                 result is exact to about 2^-16 before its own rounding.
// The running maximum of the softmax is only raised when a score passes it by
// 2^24 (BF16 and fp32 hold that without loss), so that a tile costs a vote
// in place of shuffles.
#include <cmath>

#include "kernels.h"
#include "kv4_attn.cuh"
#include "kv4_host.h"
#include "tc.cuh"

namespace uw {

namespace {

constexpr int kWarps = 8;
constexpr int kTile = 32;            // keys of a unit
constexpr float kRaise = 24.f;       // log2 headroom of a probability
constexpr uint32_t kWholeUnits = 32; // items up to this many units are not cut while shares are short

template <int D>
constexpr int kStageBytes = kTile * (D + 8);
template <int D>
constexpr int kStages = D == 128 ? 3 : 5;

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// 16 + c for the codes in bits 3..6 of both halves: the upper four of a
// BF16's seven mantissa bits at 2^4.
__device__ __forceinline__ uint32_t code_pair(uint32_t w) { return (w & 0x00780078u) | 0x41804180u; }
// The same less 24: c - 8 (exact).
__device__ __forceinline__ uint32_t centred_pair(uint32_t w) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(code_pair(w)), "r"(0x41c041c0u));
    return r;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The key of a tile that row k of a product's 16 stands for: with rows 2, 3
// (mod 4) exchanged, the eight rows of a K load and the rows that a V load
// takes from one lane group fall on different halves of the banks.
__device__ __forceinline__ int key_of(int k) { return k ^ ((k >> 1) & 1); }

// Where 16-byte chunk ch of V row r lies in its row (D = 128: rows 4..7 of
// eight have their halves exchanged, against bank conflicts of the 8-byte loads).
template <int D>
__device__ __forceinline__ int v_chunk(int r, int ch) {
    return D == 128 ? ch ^ (((r >> 2) & 1) << 1) : ch;
}

// Where float4 c of a row lies in a warp's part: the four pairs of rows that
// are written together exchange their places against bank conflicts.
template <int D>
__device__ __forceinline__ int part_at(int row, int c) {
    constexpr int N = D / 32;
    return row * (D / 4) + (c ^ (((row & 7) >> 1) & (N - 1)));
}

template <int D, int NT>
struct Warp {
    // D/16 pairs of dimensions of the output for 2 rows of each of NT row groups
    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2], z[NT][2];
    uint32_t q[NT][D / 16][2];
    float qs[NT][2];
};

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 2 : 1) kv4_decode_kernel(const AttnParams p) {
    constexpr int RB = 8 * NT;
    constexpr int ST = kStages<D>;
    using S = Sched<RB, kTile>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t slots[kWarps];
    __shared__ uint64_t found_base[2];
    __shared__ int found_seq[2];
    __shared__ float w_m[kWarps][RB], w_l[kWarps][RB];
    __shared__ uint32_t arrived;
    grid_dep_launch();
    grid_dep_wait();
    const Kv4View &v = p.v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * ST * kStageBytes<D>;

    // this CTA's share [ua, ub) of the units, and where it begins
    const int per = (v.n_seqs + kWarps * 32 - 1) / (kWarps * 32);
    const int sa = min(int(threadIdx.x) * per, v.n_seqs), sb = min(sa + per, v.n_seqs);
    uint64_t mine = 0;
    for (int s = sa; s < sb; s++)
        mine += S::seq_units(p, kv4_seq(v, s)) * v.heads;
    uint64_t total;
    const uint64_t before = cta_prefix<kWarps * 32>(mine, slots, &total);
    const uint32_t workers = uint32_t(min(total, uint64_t(gridDim.x)));
    if (blockIdx.x >= workers)
        return;
    uint64_t cut[2] = {total * blockIdx.x / workers, total * (blockIdx.x + 1) / workers};
    for (int k = 0; k < 2; k++)
        if (before <= cut[k] && cut[k] < before + mine) {
            uint64_t u = before;
            for (int s = sa; s < sb; s++) {
                const uint64_t w = S::seq_units(p, kv4_seq(v, s)) * v.heads;
                if (cut[k] < u + w) {
                    found_seq[k] = s;
                    found_base[k] = u;
                    break;
                }
                u += w;
            }
        }
    __syncthreads();
    auto locate = [&](int k) {
        Item it;
        it.s = found_seq[k];
        it.q = kv4_seq(v, it.s);
        const uint64_t per_head = S::seq_units(p, it.q);
        uint64_t rest = cut[k] - found_base[k];
        it.head = int(rest / per_head);
        rest -= it.head * per_head;
        it.u0 = found_base[k] + it.head * per_head;
        for (it.rt = 0;; it.rt++) {
            it.keys = S::tile_keys(p, it.q, it.rt);
            it.n = S::units(it.keys);
            if (rest < it.n)
                break;
            rest -= it.n;
            it.u0 += it.n;
        }
        return it;
    };
    // While a share is at most a tile for each warp, an item of a few tiles
    // a warp is taken whole: a cut through it would cost a round trip through
    // the workspace.
    const bool whole = total <= uint64_t(kWarps) * gridDim.x;
    Item it = locate(0);
    if (whole && it.n <= kWholeUnits)
        cut[0] = it.u0;
    if (cut[1] < total) {
        const Item e = locate(1);
        if (whole && e.n <= kWholeUnits)
            cut[1] = e.u0;
    }

    uint64_t u = cut[0];
    while (u < cut[1]) {
        const uint32_t seg_a = uint32_t(u - it.u0), seg_b = uint32_t(min(cut[1] - it.u0, uint64_t(it.n)));
        const int tile0 = it.keys.lo / kTile;
        const bool some = it.keys.hi > it.keys.lo;
        const int tiles = some ? int(seg_b - seg_a) : 0;
        const int first = tile0 + int(seg_a) + warp;       // this warp's tiles: first, first + kWarps, ...
        const int n_mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
        const int64_t r0 = int64_t(it.rt) * RB;
        const int64_t rows = int64_t(it.q.n) * p.group;
        // keys that every row of the item sees
        const int tok_a = int(r0 / p.group), tok_b = int((min(r0 + RB, rows) - 1) / p.group);
        const KeyRange ka = visible(p, it.q, tok_a, tok_a), kb = visible(p, it.q, tok_b, tok_b);
        const int all_lo = kb.lo, all_hi = min(ka.hi, it.q.len);

        // A tile's copies.  The lane's page is that of key 16 * (lane / 16) of the tile.
        auto page_of = [&](int tile) -> int {
            const int key = tile * kTile + (lane & 16);
            if (key >= it.q.len)
                return -1;
            const int page = __ldg(v.table + int64_t(it.s) * v.table_stride + (key >> v.page_log2));
            if (uint32_t(page) >= uint64_t(v.n_pages)) {
                atomicOr(v.status, uint32_t(kStatusBadCache));
                return -1;
            }
            return page;
        };
        const int64_t block = int64_t(D + 8) << v.page_log2;
        const int mask = (1 << v.page_log2) - 1;
        auto issue = [&](int tile, int page, int stage) {
            const uint32_t dst = ring + stage * kStageBytes<D>;
            const int key0 = tile * kTile;
            const uint8_t *const base = v.pages + it.head * block;
            constexpr int RC = D / 32;             // 16-byte chunks of a row
            constexpr int RPI = 32 / RC;           // rows of one instruction
#pragma unroll
            for (int j = 0; j < RC; j++) {
                const int r = j * RPI + lane / RC, ch = lane % RC;
                const int pg = __shfl_sync(0xffffffffu, page, r & 16);
                const bool in = pg >= 0 && key0 + r < it.q.len;
                const uint8_t *src = in ? base + pg * (block * v.heads) + ((key0 + r) & mask) * (D / 2) + ch * 16 : v.pages;
                cp_async16_zfill(dst + r * (D / 2) + ch * 16, src, in ? 16u : 0u);
                src = in ? src + ((D / 2) << v.page_log2) : v.pages;
                cp_async16_zfill(dst + kTile * (D / 2) + r * (D / 2) + v_chunk<D>(r, ch) * 16, src, in ? 16u : 0u);
            }
            const int r = (lane & 7) * 4, is_v = (lane >> 3) & 1;
            const int pg = __shfl_sync(0xffffffffu, page, r & 16);
            if (lane < 16) {
                const bool in = pg >= 0 && key0 + r < it.q.len;
                const uint8_t *src = in ? base + pg * (block * v.heads) +
                                              kv4_params<D>(v.page_log2, (key0 + r) & mask, is_v)
                                        : v.pages;
                cp_async16_zfill(dst + kTile * D + is_v * (kTile * 4) + r * 4, src, in ? 16u : 0u);
            }
        };
        int page_next = n_mine > 0 ? page_of(first) : -1;
#pragma unroll
        for (int s = 0; s < ST - 1; s++) {
            const int page = page_next;
            if (s + 1 < n_mine)
                page_next = page_of(first + (s + 1) * kWarps);
            if (s < n_mine)
                issue(first + s * kWarps, page, s);
            cp_async_commit();
        }

        Warp<D, NT> w;
        // Queries: lane (g, t) holds row g of each group, dimensions D/4 t .. + D/4 - 1,
        // paired as the codes of a word come out of it: (0,4) (1,5) (2,6) (3,7).
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int64_t r = r0 + nt * 8 + g;
            uint4 x[D / 32];
#pragma unroll
            for (int k = 0; k < D / 32; k++)
                x[k] = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const int64_t tok = it.q.t0 + r / p.group, head = int64_t(it.head) * p.group + r % p.group;
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q.p + tok * p.q.ts + head * p.q.hs + (D / 4) * t);
#pragma unroll
                for (int k = 0; k < D / 32; k++)
                    x[k] = src[k];
            }
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < D / 32; k++) {
                w.q[nt][2 * k][0] = __byte_perm(x[k].x, x[k].z, 0x5410);
                w.q[nt][2 * k][1] = __byte_perm(x[k].x, x[k].z, 0x7632);
                w.q[nt][2 * k + 1][0] = __byte_perm(x[k].y, x[k].w, 0x5410);
                w.q[nt][2 * k + 1][1] = __byte_perm(x[k].y, x[k].w, 0x7632);
                const uint32_t a[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int i = 0; i < 4; i++)
                    sum += bf16_lo(a[i]) + bf16_hi(a[i]);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            w.qs[nt][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
            w.qs[nt][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
#pragma unroll
            for (int k = 0; k < 2; k++) {
                w.m[nt][k] = -INFINITY;
                w.l[nt][k] = w.z[nt][k] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < D / 16; i++)
#pragma unroll
                for (int k = 0; k < 4; k++)
                    w.o[i][nt][k] = 0.f;
        }

        for (int i = 0; i < n_mine; i++) {
            {
                const int nx = i + ST - 1;
                const int page = page_next;
                if (nx + 1 < n_mine)
                    page_next = page_of(first + (nx + 1) * kWarps);
                if (nx < n_mine)
                    issue(first + nx * kWarps, page, nx % ST);
                cp_async_commit();
            }
            asm volatile("cp.async.wait_group %0;" :: "n"(ST - 1) : "memory");
            __syncwarp();
            const uint32_t st = ring + (i % ST) * kStageBytes<D>;
            const int key0 = (first + i * kWarps) * kTile;

            // scores
            float sc[2][NT][4];
#pragma unroll
            for (int mt = 0; mt < 2; mt++) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        sc[mt][nt][k] = 0.f;
                uint32_t a[D / 32], b[D / 32];
                const uint32_t row = st + (16 * mt + key_of(g)) * (D / 2) + t * (D / 8);
                if constexpr (D == 128) {
                    const uint4 x = lds128(row), y = lds128(row + 8 * (D / 2));
                    a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
                    b[0] = y.x, b[1] = y.y, b[2] = y.z, b[3] = y.w;
                } else {
                    const uint2 x = lds64(row), y = lds64(row + 8 * (D / 2));
                    a[0] = x.x, a[1] = x.y;
                    b[0] = y.x, b[1] = y.y;
                }
#pragma unroll
                for (int k = 0; k < D / 32; k++)
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const uint32_t a0 = code_pair(j ? a[k] >> 5 : a[k] << 3);
                        const uint32_t a1 = code_pair(j ? b[k] >> 5 : b[k] << 3);
                        const uint32_t a2 = code_pair(j ? a[k] >> 9 : a[k] >> 1);
                        const uint32_t a3 = code_pair(j ? b[k] >> 9 : b[k] >> 1);
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
                            mma16816(sc[mt][nt], a0, a1, a2, a3, w.q[nt][2 * k + j][0], w.q[nt][2 * k + j][1]);
                    }
            }
            // sc[mt][nt][2 h + k]: key 16 mt + 8 h + key_of(g), row 8 nt + 2 t + k
            uint32_t vpar[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t at = st + kTile * D + (8 * j + key_of(g)) * 4;
                const uint32_t kp = lds32(at);
                vpar[j] = lds32(at + kTile * 4);
                const float a = bf16_lo(kp) * p.c1, c = fmaf(bf16_hi(kp), p.c1, -16.f * a);
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        float &y = sc[j >> 1][nt][2 * (j & 1) + k];
                        y = fmaf(y, a, c * w.qs[nt][k]);
                    }
            }
            const bool open = key0 < all_lo || key0 + kTile > all_hi;
            if (open) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const int64_t r = min(r0 + nt * 8 + 2 * t + k, rows - 1);
                        const int tok = int(r / p.group);
                        const KeyRange kr = visible(p, it.q, tok, tok);
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const int key = key0 + 8 * j + key_of(g);
                            if (key < kr.lo || key >= min(kr.hi, it.q.len))
                                sc[j >> 1][nt][2 * (j & 1) + k] = -INFINITY;
                        }
                    }
            }
            // raise the maximum where a score passes it by far
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const float top = fmaxf(fmaxf(sc[0][nt][k], sc[0][nt][2 + k]), fmaxf(sc[1][nt][k], sc[1][nt][2 + k]));
                    raise = raise || top > w.m[nt][k] + kRaise;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        float top = fmaxf(fmaxf(sc[0][nt][k], sc[0][nt][2 + k]), fmaxf(sc[1][nt][k], sc[1][nt][2 + k]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const float m2 = fmaxf(w.m[nt][k], top);
                        const float f = m2 == -INFINITY ? 1.f : exp2_fast(w.m[nt][k] - m2);
                        w.m[nt][k] = m2;
                        w.l[nt][k] *= f;
                        w.z[nt][k] *= f;
#pragma unroll
                        for (int d = 0; d < D / 16; d++) {
                            w.o[d][nt][k] *= f;
                            w.o[d][nt][2 + k] *= f;
                        }
                    }
            }
            // probabilities, as the B operand of the product with V: p s in two BF16
            uint32_t hi[2][NT][2], lo[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const float m0 = w.m[nt][0] == -INFINITY ? 0.f : w.m[nt][0];
                const float m1 = w.m[nt][1] == -INFINITY ? 0.f : w.m[nt][1];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float s = bf16_lo(vpar[j]), mid = fmaf(8.f, s, bf16_hi(vpar[j]));
                    const float y0 = sc[j >> 1][nt][2 * (j & 1)], y1 = sc[j >> 1][nt][2 * (j & 1) + 1];
                    const float p0 = exp2_fast(y0 - m0), p1 = exp2_fast(y1 - m1);
                    w.l[nt][0] += p0;
                    w.l[nt][1] += p1;
                    float s0 = p0 * s, s1 = p1 * s, z0 = p0 * mid, z1 = p1 * mid;
                    if (open) {  // a masked key's scale may be anything
                        s0 = y0 == -INFINITY ? 0.f : s0;
                        s1 = y1 == -INFINITY ? 0.f : s1;
                        z0 = y0 == -INFINITY ? 0.f : z0;
                        z1 = y1 == -INFINITY ? 0.f : z1;
                    }
                    w.z[nt][0] += z0;
                    w.z[nt][1] += z1;
                    const uint32_t h = bf16_pack(s0, s1);
                    hi[j >> 1][nt][j & 1] = transpose8x8(h);
                    lo[j >> 1][nt][j & 1] = transpose8x8(bf16_pack(s0 - bf16_lo(h), s1 - bf16_hi(h)));
                }
            }
            // output
#pragma unroll
            for (int mt = 0; mt < 2; mt++) {
                constexpr int VW = D / 64;  // 32-bit words of a row for one lane
                uint32_t x[4][VW];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    // keys of the product's rows 2t, 2t + 1, 2t + 8, 2t + 9
                    const int r = 16 * mt + 8 * (j >> 1) + key_of(2 * t + (j & 1));
                    const uint32_t base = st + kTile * (D / 2) + r * (D / 2);
                    if constexpr (D == 128) {
                        const uint2 y = lds64(base + v_chunk<D>(r, g >> 1) * 16 + (g & 1) * 8);
                        x[j][0] = y.x, x[j][1] = y.y;
                    } else {
                        x[j][0] = lds32(base + g * 4);
                    }
                }
#pragma unroll
                for (int k = 0; k < VW; k++)
#pragma unroll
                    for (int b = 0; b < 4; b++) {
                        const uint32_t sel = b * 0x11u | (4 + b) * 0x1100u;
                        const uint32_t e = __byte_perm(x[0][k], x[1][k], sel), f = __byte_perm(x[2][k], x[3][k], sel);
                        const uint32_t a0 = centred_pair(e << 3), a1 = centred_pair(e >> 1);
                        const uint32_t a2 = centred_pair(f << 3), a3 = centred_pair(f >> 1);
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) {
                            mma16816(w.o[4 * k + b][nt], a0, a1, a2, a3, hi[mt][nt][0], hi[mt][nt][1]);
                            mma16816(w.o[4 * k + b][nt], a0, a1, a2, a3, lo[mt][nt][0], lo[mt][nt][1]);
                        }
                    }
            }
            __syncwarp();
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");

        // The warps' parts, joined through shared memory: each warp leaves its
        // maximum, sum and output (with the ranges' middles added) in its own ring.
        float4 *const wo = reinterpret_cast<float4 *>(smem + warp * ST * kStageBytes<D>);
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int k = 0; k < 2; k++) {
                float l = w.l[nt][k], z = w.z[nt][k];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    l += __shfl_xor_sync(0xffffffffu, l, o);
                    z += __shfl_xor_sync(0xffffffffu, z, o);
                }
                const int row = 8 * nt + 2 * t + k;
                if (g == 0) {
                    w_m[warp][row] = w.m[nt][k];
                    w_l[warp][row] = l;
                }
                // dimensions D/8 g .. + D/8 - 1 of this row
#pragma unroll
                for (int i = 0; i < D / 32; i++)
                    wo[part_at<D>(row, g * (D / 32) + i)] =
                        make_float4(w.o[2 * i][nt][k] + z, w.o[2 * i][nt][2 + k] + z, w.o[2 * i + 1][nt][k] + z,
                                    w.o[2 * i + 1][nt][2 + k] + z);
            }
        __syncthreads();

        // This part's place among the item's, and the item's output once all are there.
        const uint32_t f = share_of(it.u0, total, workers), e = share_of(it.u0 + it.n - 1, total, workers);
        const bool alone = seg_a == 0 && seg_b == it.n;
        constexpr int F4 = RB * (D / 4);
        float *const part = p.parts + (2 * uint64_t(blockIdx.x) + (seg_a == 0 ? 1 : 0)) * (RB * (D + 2));
        for (int x = threadIdx.x; x < F4; x += kWarps * 32) {
            const int row = x / (D / 4), c = x % (D / 4);
            float m = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWarps; k++)
                m = fmaxf(m, w_m[k][row]);
            const float m0 = m == -INFINITY ? 0.f : m;
            float l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; k++) {
                const float fw = exp2_fast(w_m[k][row] - m0);
                const float4 o = reinterpret_cast<const float4 *>(smem + k * ST * kStageBytes<D>)[part_at<D>(row, c)];
                l = fmaf(fw, w_l[k][row], l);
                acc.x = fmaf(fw, o.x, acc.x);
                acc.y = fmaf(fw, o.y, acc.y);
                acc.z = fmaf(fw, o.z, acc.z);
                acc.w = fmaf(fw, o.w, acc.w);
            }
            if (alone) {
                store_row<D>(p, it, r0 + row, rows, c, acc, m, l);
            } else {
                reinterpret_cast<float4 *>(part)[x] = acc;
                if (c == 0) {
                    part[RB * D + row] = m;
                    part[RB * D + RB + row] = l;
                }
            }
        }
        if (!alone) {
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                arrived = atomicAdd(p.counters + f, 1u) == e - f;
                if (arrived)
                    p.counters[f] = 0;  // ready for the next call
            }
            __syncthreads();
            if (arrived) {
                __threadfence();
                for (int x = threadIdx.x; x < F4; x += kWarps * 32) {
                    const int row = x / (D / 4), c = x % (D / 4);
                    float m = -INFINITY, l = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (uint32_t k = f; k <= e; k++) {
                        const float *q = p.parts + (2 * uint64_t(k) + (k == f ? 1 : 0)) * (RB * (D + 2));
                        join(m, l, acc, __ldcg(q + RB * D + row), __ldcg(q + RB * D + RB + row),
                             __ldcg(reinterpret_cast<const float4 *>(q) + x));
                    }
                    store_row<D>(p, it, r0 + row, rows, c, acc, m, l);
                }
            }
        }
        __syncthreads();  // the rings are free again

        u += seg_b - seg_a;
        if (u < cut[1]) {
            it.u0 += it.n;
            if (++it.rt == S::row_tiles(p, it.q)) {
                it.rt = 0;
                if (++it.head == v.heads) {
                    it.head = 0;
                    do
                        it.q = kv4_seq(v, ++it.s);
                    while (!S::mine(p, it.q));
                }
            }
            it.keys = S::tile_keys(p, it.q, it.rt);
            it.n = S::units(it.keys);
        }
    }
}

template <int D, int NT>
uw_status launch(const AttnParams &p, int ctas, cudaStream_t st) {
    constexpr size_t smem = size_t(kWarps) * kStages<D> * kStageBytes<D>;
    if (!ensure_smem(kv4_decode_kernel<D, NT>, smem))
        return UW_ERR_CUDA;
    return launch_overlapped(kv4_decode_kernel<D, NT>, dim3(unsigned(ctas)), dim3(kWarps * 32), smem, st, p) ==
                   cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}

}  // namespace

int kv4_decode_ctas() { return 2 * sm_count(); }

size_t kv4_decode_part_floats(int head_dim) { return 2 * size_t(kv4_decode_ctas()) * 16 * (head_dim + 2); }

// Eight rows a tile where no sequence has more (one new token of up to eight
// heads a group), sixteen otherwise.
uw_status launch_kv4_decode(const AttnParams &p, int head_dim, int64_t rows, int64_t max_units, cudaStream_t st) {
    const bool wide = rows == 0 || rows > 8;
    int64_t ctas = wide ? kv4_decode_ctas() / 2 : kv4_decode_ctas();
    if (max_units > 0)
        ctas = std::min(ctas, max_units);
    const int n = int(ctas);
    if (head_dim == 128)
        return wide ? launch<128, 2>(p, n, st) : launch<128, 1>(p, n, st);
    return wide ? launch<64, 2>(p, n, st) : launch<64, 1>(p, n, st);
}

}  // namespace uw
