// Attention over keys and values as they were projected (BF16 rows, no cache): whole
// sequences of different lengths behind each other, grouped heads.
//
// The floor is the tensor cores'.  One persistent CTA an SM takes an equal share of all
// (256 rows x 128 keys) steps (attn_work.cuh); a row is a query head of a token, rows of one
// kv head lie together, so a tile of K and V is read once for all of them.  Warp roles:
//   softmax   warps 0-3 and 4-7: the upper and lower 128 rows, a row a thread.  They read
//             S from tensor memory, take the exponentials and write P (BF16) over S, where
//             the second product reads it; at the end of an item they write the rows' output.
//   helper    warps 8-11: the queries of an item into shared memory, in a ring of three
//             halves, so that those of the next item come in beside this one; V of tiles that
//             some row does not see in full (see below).
//   MMA       warps 12 and 13, for the upper and lower rows, one elected thread each (a
//             thread takes some 50 cycles for each product that it issues and 140 for a wait, 3500 a
//             step for both halves): S = Q K^T and O += P V with tcgen05.mma, 128 rows and 128 keys
//             each; while the softmax works on one half of the rows, the products of the other
//             half run.
//   copies    warp 14, one elected thread: tiles of K and V by tensor-map copies, two
//             stages of each.  V lies as it comes, [keys][dims], and is the second product's
//             operand with its rows along the product.
// The running maximum is only raised when some row's probabilities of a tile add up to
// more than 2^24 (BF16 and fp32 hold that without loss), so that after the first keys no score
// is compared and O is rarely rescaled.  P is rounded to one BF16 (2^-8, the one rounding beside
// the output's); its sum is fp32 of the unrounded values.
//
// What a row does not see takes no part in it, whatever its bits: a masked score is
// replaced before its exponential, and since 0 times a V that is not finite is not 0, the
// helper looks through V's tiles that are not seen by all rows, zeroes keys past the sequence's
// end and values that are not finite, and an item with such a value adds them at its end to the rows
// that see their keys.
#include <cudaTypedefs.h>

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "attn_work.cuh"
#include "kernels.h"
#include "kv4_host.h"
#include "tmem.cuh"

namespace uw {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // gemm_tc.cu

namespace {

constexpr int kRows = 256, kKeys = 128;
constexpr int kSoftmax = 256, kHelper = 128;          // threads
constexpr int kThreads = kSoftmax + kHelper + 128;    // and a warpgroup of the MMA and copying warps
constexpr int kItemCost = 3;                          // what an item costs beyond its steps, in steps
constexpr int kMinShare = 4;                          // units of a CTA at least
constexpr int kSegs = 16;
constexpr int kStages = 2, kQSlots = 3;
constexpr float kRaise = 16777216.f;                  // 2^24: headroom of the sum of a tile's probabilities
constexpr uint32_t kTmemCols = 512;

// The call's sequences: tokens start[s] .. and keys kstart[s] ..
struct PackedView {
    const int32_t *start, *kstart;
    int64_t n_tokens, n_keys;
    int32_t n_seqs, heads;
    uint32_t *status;
};
__device__ __forceinline__ Seq seq_of(const PackedView &v, int s) {
    const int32_t a = __ldg(v.start + s), b = __ldg(v.start + s + 1), ka = __ldg(v.kstart + s),
                  kb = __ldg(v.kstart + s + 1);
    if (a < 0 || b < a || b > v.n_tokens || ka < 0 || kb < ka || kb > v.n_keys) {
        atomicOr(v.status, kStatusBadCache);
        return {0, 0, 0};
    }
    return {a, b - a, kb - ka};
}

struct PackedParams {
    PackedView v;
    Rows q, o, val;
    float *lse;
    float c1;                    // softmax scale * log2(e)
    int32_t q_heads, group, causal, window;
    Divisor by_group;
    bool out32;                  // rows of o begin on 32-byte steps
    bool heads_outer[2], one_head[2];  // of K, V: the tensor map's outermost dimension is the head; all heads are one
    int32_t rows_min, rows_max;  // any
    float *parts;                // parts of kRows * (D + 2) floats: output, maximum, sum
    uint32_t *counters;          // [gridDim.x], left at zero
    CUtensorMap kmap, vmap;      // 64 dimensions x 128 keys of one head
};

enum Bar {
    kQFull, kQEmpty = kQFull + kQSlots, kKFull = kQEmpty + kQSlots, kKEmpty = kKFull + kStages, kVFull = kKEmpty + kStages, kVOk = kVFull + kStages,
    kVEmpty = kVOk + kStages, kTurn = kVEmpty + kStages, kSFull = kTurn + 2, kPFull = kSFull + 2, kPvDone = kPFull + 2,
    kBars = kPvDone + 2
};

struct Shared {
    uint64_t bars[kBars];
    uint64_t listed_to;
    Seg segs[kSegs];
    int32_t key0[kSegs];   // the sequence's first key
    uint32_t hurt[kSegs];  // V of a tile that not all rows see holds a value that is not finite
    uint32_t tmem, dead, arrived;
    int n_segs;
};

template <int D>
constexpr uint32_t kTileBytes = kKeys * D * 2;  // 128 rows of Q, 128 keys of K or V
template <int D>
constexpr size_t kSmem = 1024 + (kQSlots + 2 * kStages) * size_t(kTileBytes<D>);

// A wait that every thread of a role makes at the same place.  One that runs
// out marks the kernel dead: all later waits return at once, every role
// walks through its remaining steps without waiting, and the status word tells.
__device__ __forceinline__ bool is_dead(Shared &sh) { return *reinterpret_cast<volatile uint32_t *>(&sh.dead) != 0; }
__device__ __forceinline__ void wait(Shared &sh, uint32_t bar, uint32_t parity, uint32_t *status) {
    if (mbar_try_wait(bar, parity) || is_dead(sh))
        return;
    if (!mbar_wait(bar, parity, status, kStatusTimeout))
        *reinterpret_cast<volatile uint32_t *>(&sh.dead) = 1;
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Byte offset of 16-byte chunk c (8 values) of row r in a tile of 128 rows:
// blocks of 64 values, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    return uint32_t(c >> 3) * (128u * 128u) + sw128_offset(uint32_t(r), uint32_t(c & 7));
}

// Whether some row of the segment does not see some key of the tile at key0.
__device__ __forceinline__ bool is_open(const Seg &sg, int key0) {
    return key0 < sg.all_lo || sg.all_hi - key0 < kKeys;  // (key0 + kKeys may be 2^31)
}

// All of the thread's groups of copies but the last are done.
__device__ __forceinline__ void cp_async_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

__device__ __forceinline__ bool not_finite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// A value that is the same in all lanes, so that what follows from it stays in uniform
// registers, which the products' descriptors and addresses are taken from.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

template <int D>
__device__ __forceinline__ void mma_role(const PackedParams &p, Shared &sh, uint32_t bars, uint32_t q_at,
                                         uint32_t k_at, uint32_t v_at, int half, uint32_t &steps, uint32_t &cnt,
                                         uint32_t &halves, uint32_t &turns) {
    constexpr uint32_t kIdS = idesc_bf16_f32(128, kKeys), kIdO = idesc_bf16_f32(128, D) | kTransposeB;
    const uint32_t tm = uint32_t(uniform(int(sh.tmem))), s_tm = tm + half * kKeys, o_tm = tm + 256 + half * D;
    // Descriptors of the tiles; a step of 16 values along the first product adds 32
    // bytes, the next block of 64 values 128 * 128, a step of 16 keys along the second 16 * 128.
    const uint64_t q_desc = sdesc_sw128(q_at), k_desc = sdesc_sw128(k_at), v_desc = sdesc_sw128_n(v_at, 128 * 128);
    auto at = [](int i) { return uint64_t((i / 4) * (128 * 8) + (i % 4) * 2); };
    const int n_segs = uniform(sh.n_segs);
    for (int s = 0; s < n_segs; s++) {
        const Seg &sg = sh.segs[s];
        const int tiles = uniform(sg.tiles), rows = uniform(sg.tokens * p.group - sg.rt * kRows);
        if (tiles == 0)
            continue;
        const bool two = rows > 128, active = half == 0 || two;
        const uint32_t slot = (halves + half) % kQSlots;
        // The halves take turns, each with its outputs and next scores, so that one half's products
        // run while the other's softmax does (without turns both end up at the same place).
        auto my_turn = [&]() {
            if (two)
                wait(sh, bars + 8 * (kTurn + half), (turns & 1) ^ (half ^ 1), p.v.status);
        };
        auto pass = [&]() {  // by the elected thread
            if (two)
                mbar_arrive(bars + 8 * (kTurn + (half ^ 1)));
        };
        // Step j's scores behind step j - 1's outputs: S lies over P.
        for (int j = 0; j <= tiles; j++) {
            const uint32_t step = steps + j, before = step - 1, k_stage = step % kStages, v_stage = before % kStages;
            if (j > 0)
                wait(sh, bars + 8 * (kVOk + v_stage), (before / kStages) & 1, p.v.status);
            if (!active) {
                if (j > 0 && elect_one())
                    mbar_arrive(bars + 8 * (kVEmpty + v_stage));
                if (j < tiles) {
                    wait(sh, bars + 8 * (kKFull + k_stage), (step / kStages) & 1, p.v.status);
                    if (elect_one())
                        mbar_arrive(bars + 8 * (kKEmpty + k_stage));
                }
                continue;
            }
            // (a wait takes 140 cycles, done or not: the probabilities', which all else waits for, comes last)
            if (j < tiles)
                wait(sh, bars + 8 * (kKFull + k_stage), (step / kStages) & 1, p.v.status);
            if (j == 0)
                wait(sh, bars + 8 * (kQFull + slot), ((halves + half) / kQSlots) & 1, p.v.status);
            my_turn();
            turns += two;
            if (j > 0)
                wait(sh, bars + 8 * (kPFull + half), cnt++ & 1, p.v.status);
            tc_fence_after();
            if (elect_one()) {
                if (j > 0) {
                    const uint64_t v = v_desc + v_stage * (kTileBytes<D> >> 4);
#pragma unroll
                    for (int i = 0; i < kKeys / 16; i++)
                        mma_ts(o_tm, s_tm + 8 * i, v + i * (16 * 8), kIdO, j > 1 || i > 0);
                    mma_commit(bars + 8 * (kPvDone + half));
                    mma_commit(bars + 8 * (kVEmpty + v_stage));
                }
                if (j < tiles) {
                    const uint64_t q = q_desc + slot * (kTileBytes<D> >> 4), k = k_desc + k_stage * (kTileBytes<D> >> 4);
#pragma unroll
                    for (int i = 0; i < D / 16; i++)
                        mma_bf16(s_tm, q + at(i), k + at(i), kIdS, i > 0);
                    mma_commit(bars + 8 * (kSFull + half));
                    mma_commit(bars + 8 * (kKEmpty + k_stage));
                    if (j == tiles - 1)
                        mma_commit(bars + 8 * (kQEmpty + slot));
                }
                pass();
            }
            __syncwarp();
        }
        steps += tiles;
        halves += two ? 2 : 1;
    }
    // every commit has arrived before the barriers go
    if (steps > 0)
        wait(sh, bars + 8 * (kVEmpty + (steps - 1) % kStages), ((steps - 1) / kStages) & 1, p.v.status);
}

template <int D>
__device__ __forceinline__ void copy_role(const PackedParams &p, Shared &sh, uint32_t bars, uint32_t k_at,
                                          uint32_t v_at, uint32_t &steps) {
    auto copy = [&](const CUtensorMap &map, int which, uint32_t to, int head, int key, uint32_t bar) {
        head = p.one_head[which] ? 0 : head;
        mbar_expect_tx(bar, kTileBytes<D>);
#pragma unroll
        for (int b = 0; b < D / 64; b++)
            tma_load_3d(to + b * (128 * 128), &map, 64 * b, p.heads_outer[which] ? key : head,
                        p.heads_outer[which] ? head : key, bar);
    };
    // What is on its way ends before the CTA does, whatever became of the rest: n tiles of K, n - less of V.
    auto drain = [&](uint32_t n, uint32_t less) {
        for (uint32_t i = n - min(n, uint32_t(kStages)); i < n; i++) {
            mbar_wait(bars + 8 * (kKFull + i % kStages), (i / kStages) & 1, p.v.status, kStatusTimeout);
            if (i + less < n)
                mbar_wait(bars + 8 * (kVFull + i % kStages), (i / kStages) & 1, p.v.status, kStatusTimeout);
        }
    };
    for (int s = 0; s < sh.n_segs; s++) {
        const Seg &sg = sh.segs[s];
        for (int j = 0; j < sg.tiles; j++, steps++) {
            const uint32_t stage = steps % kStages, free = ((steps / kStages) & 1) ^ 1;
            const int key = sh.key0[s] + (sg.first + j) * kKeys;
            wait(sh, bars + 8 * (kKEmpty + stage), free, p.v.status);
            if (is_dead(sh))
                return drain(steps, 0);
            copy(p.kmap, 0, k_at + stage * kTileBytes<D>, sg.head, key, bars + 8 * (kKFull + stage));
            wait(sh, bars + 8 * (kVEmpty + stage), free, p.v.status);
            if (is_dead(sh))
                return drain(steps + 1, 1);
            copy(p.vmap, 1, v_at + stage * kTileBytes<D>, sg.head, key, bars + 8 * (kVFull + stage));
        }
    }
}

template <int D>
__device__ __forceinline__ void helper_role(const PackedParams &p, Shared &sh, uint32_t bars, uint32_t q_at,
                                            uint32_t v_at, uint32_t &steps, uint32_t &halves) {
    constexpr int C = D / 8;  // 16-byte chunks of a row
    const int t = threadIdx.x - kSoftmax, lane = t & 31;
    for (int s = 0; s < sh.n_segs; s++) {
        const Seg &sg = sh.segs[s];
        if (sg.tiles == 0)
            continue;
        const int r0 = sg.rt * kRows, rows = min(sg.tokens * p.group - r0, kRows), two = rows > 128;
        for (int half = 0; half <= two; half++) {
            const uint32_t slot = (halves + half) % kQSlots;
            wait(sh, bars + 8 * (kQEmpty + slot), (((halves + half) / kQSlots) & 1) ^ 1, p.v.status);
#pragma unroll 4
            for (int x = t; x < 128 * C; x += kHelper) {
                const int rr = x / C, c = x % C;
                const bool in = 128 * half + rr < rows;
                const int r = r0 + (in ? 128 * half + rr : 0), i = p.by_group.of(r);
                cp_async16_zfill(q_at + slot * kTileBytes<D> + tile_at(rr, c),
                                 p.q.p + (sg.t0 + int64_t(i)) * p.q.ts +
                                     (sg.head * p.group + (r - i * p.group)) * p.q.hs + 8 * c,
                                 in ? 16 : 0);
            }
            cp_async_commit();
        }
        for (int half = 0; half <= two; half++) {
            if (half < two)
                cp_async_wait_but_one();
            else
                cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bars + 8 * (kQFull + (halves + half) % kQSlots));
        }
        halves += 1 + two;
        for (int j = 0; j < sg.tiles; j++, steps++) {
            const uint32_t stage = steps % kStages;
            const int key0 = (sg.first + j) * kKeys;
            wait(sh, bars + 8 * (kVFull + stage), (steps / kStages) & 1, p.v.status);
            if (is_open(sg, key0)) {
                // a key a thread
                const uint32_t tile = v_at + stage * kTileBytes<D>;
                const bool there = t < sg.len - key0;
                bool hurt = false;
#pragma unroll
                for (int c = 0; c < C; c++) {
                    const uint32_t at = tile + tile_at(t, c);
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
                    bool bad = false;
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        bad = bad || not_finite(w[k]);
                    if (bad || !there) {
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const bool low = (w[k] & 0x7f80u) == 0x7f80u, high = (w[k] & 0x7f800000u) == 0x7f800000u;
                            w[k] = there ? w[k] & ((low ? 0u : 0xffffu) | (high ? 0u : 0xffff0000u)) : 0u;
                        }
                        sts128(at, w[0], w[1], w[2], w[3]);
                        hurt = hurt || (bad && there);
                    }
                }
                if (hurt)
                    *reinterpret_cast<volatile uint32_t *>(&sh.hurt[s]) = 1;
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bars + 8 * (kVOk + stage));
        }
    }
}

template <int D>
__device__ __forceinline__ void softmax_role(const PackedParams &p, Shared &sh, uint32_t bars, uint64_t total,
                                             uint32_t workers, uint64_t cut0, uint32_t &cnt) {
    constexpr int PF = kRows * (D + 2);
    const int half = threadIdx.x >> 7, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t s_tm = sh.tmem + lanes + half * kKeys, o_tm = sh.tmem + lanes + 256 + half * D;
    const uint64_t c1 = pair2(p.c1, p.c1);
    for (int sgi = 0; sgi < sh.n_segs; sgi++) {
        const Seg &sg = sh.segs[sgi];
        const int r0 = sg.rt * kRows, rows = sg.tokens * p.group;
        const int r = r0 + int(threadIdx.x);
        const bool active = r0 + 128 * half < rows;  // this half has rows
        const Seq sq{sg.t0, sg.tokens, sg.len};
        KeyRange mine{0, 0};
        if (r < rows) {
            const int i = p.by_group.of(r);
            mine = visible(p, sq, i, i);
            mine.hi = min(mine.hi, sg.len);
        }
        // The maximum; the sum of a tile's probabilities from which it is raised (any, as long as there is
        // none; never where there will be none).
        const float unset = mine.hi > mine.lo ? -1.f : INFINITY;
        float m = -INFINITY, lim = unset;
        uint64_t mm = 0, l2 = 0;          // less the maximum, and the sum, in pairs
        for (int j = 0; active && j < sg.tiles; j++) {
            const int key0 = (sg.first + j) * kKeys;
            wait(sh, bars + 8 * (kSFull + half), cnt & 1, p.v.status);
            tc_fence_after();
            auto tile = [&](auto masked) {
                constexpr bool kOpen = decltype(masked)::value;
                const int lo = mine.lo - key0, hi = mine.hi - key0;  // the row's keys of the tile
                auto seen = [&](int k) { return !kOpen || (k >= lo && k < hi); };
                // Raise the maximum to that of these keys, in rows that need it (not in others,
                // whose bits then depend on no other row): what the row has so far is scaled down.
                auto raise = [&](bool need) {
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < kKeys; c += 32) {
                        uint32_t x[32];
                        tmem_ld32(s_tm + c, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 32; k++)
                            if (seen(c + k))
                                top = fmaxf(top, __uint_as_float(x[k]));
                    }
                    const float m2 = need ? fmaxf(m, top * p.c1) : m, m20 = m2 == -INFINITY ? 0.f : m2;
                    const float f = !need ? 1.f : m == -INFINITY ? 0.f : exp2_fast(m - m20);
                    l2 = mul2(l2, pair2(f, f));
                    m = m2;
                    mm = pair2(-m20, -m20);
                    lim = m2 == -INFINITY ? unset : kRaise;
                    if (j > 0) {
                        wait(sh, bars + 8 * (kPvDone + half), (cnt - 1) & 1, p.v.status);
                        tc_fence_after();
#pragma unroll 1
                        for (int d0 = 0; d0 < D; d0 += 32) {
                            uint32_t w[32];
                            tmem_ld32(o_tm + d0, w);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; i++)
                                w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
                            tmem_st32(o_tm + d0, w);
                        }
                    }
                };
                // Scores are loaded 32 ahead of those whose exponentials are taken; returns the
                // sum of the probabilities, whose pairs come into pk.
                uint32_t pk[2][32];
                auto exps = [&]() {
                    uint32_t x[2][32];
                    uint64_t sum[2] = {0, 0};
                    tmem_ld32(s_tm, x[0]);
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        tmem_ld_wait();
                        if (c < 3)
                            tmem_ld32(s_tm + 32 * (c + 1), x[(c + 1) & 1]);
#pragma unroll
                        for (int k = 0; k < 16; k++) {
                            const uint32_t *const w = x[c & 1] + 2 * k;
                            float2 y = unpair(fma2(pair2(__uint_as_float(w[0]), __uint_as_float(w[1])), c1, mm));
                            if constexpr (kOpen) {
                                y.x = seen(32 * c + 2 * k) ? y.x : -INFINITY;
                                y.y = seen(32 * c + 2 * k + 1) ? y.y : -INFINITY;
                            }
                            const float a = exp2_fast(y.x), b = exp2_fast(y.y);
                            sum[k & 1] = add2(sum[k & 1], pair2(a, b));
                            pk[c >> 1][16 * (c & 1) + k] = bf16_pack(a, b);
                        }
                    }
                    return add2(sum[0], sum[1]);
                };
                if (j == 0)
                    raise(true);
                uint64_t sum = exps();
                const float2 f = unpair(sum);
                const bool need = j > 0 && f.x + f.y > lim;
                if (__any_sync(0xffffffffu, need)) {
                    raise(need);
                    sum = exps();
                }
                l2 = add2(l2, sum);
                tmem_st32(s_tm, pk[0]);
                tmem_st32(s_tm + 32, pk[1]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bars + 8 * (kPFull + half));
            };
            if (is_open(sg, key0))
                tile(std::true_type());
            else
                tile(std::false_type());
            cnt++;
        }

        const float2 lf = unpair(l2);
        const float l = lf.x + lf.y;
        const bool whole = sg.tiles == sg.of, valued = active && sg.tiles > 0;
        const int slot = cut0 > sg.u0 ? 0 : 1;
        float *const part = p.parts + (2 * uint64_t(blockIdx.x) + slot) * PF;
        if (valued) {
            wait(sh, bars + 8 * (kPvDone + half), (cnt - 1) & 1, p.v.status);
            tc_fence_after();
        }
        const bool hurt = valued && *reinterpret_cast<volatile uint32_t *>(&sh.hurt[sgi]) != 0;
        if (active) {
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; i++)
                    w[i] = 0;
                if (valued) {
                    tmem_ld32(o_tm + d0, w);
                    tmem_ld_wait();
                }
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; i++)
                    o[i] = __uint_as_float(w[i]);
                if (hurt) {
                    // values of V that are not finite, of the keys that the row sees in tiles that not all do
#pragma unroll 1
                    for (int j = 0; j < sg.tiles; j++) {
                        const int key0 = (sg.first + j) * kKeys;
                        if (!is_open(sg, key0))
                            continue;
#pragma unroll 1
                        for (int k = 0; k < kKeys; k++) {
                            const int key = key0 + k;
                            if (!(key >= mine.lo && key < mine.hi))
                                continue;
                            const uint4 *src = reinterpret_cast<const uint4 *>(
                                p.val.p + (sh.key0[sgi] + int64_t(key)) * p.val.ts + sg.head * p.val.hs + d0);
#pragma unroll
                            for (int c = 0; c < 4; c++) {
                                const uint4 v = __ldg(src + c);
                                const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int i = 0; i < 4; i++) {
                                    if ((a[i] & 0x7f80u) == 0x7f80u)
                                        o[8 * c + 2 * i] += bf16_lo(a[i]);
                                    if ((a[i] & 0x7f800000u) == 0x7f800000u)
                                        o[8 * c + 2 * i + 1] += bf16_hi(a[i]);
                                }
                            }
                        }
                    }
                }
                if (r < rows) {
                    if (whole) {
                        store_dims<32>(p, sg.t0, sg.head, r, d0, o, m, l);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            reinterpret_cast<float4 *>(part)[(d0 / 4 + i) * kRows + threadIdx.x] =
                                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
            }
            if (!whole) {
                part[kRows * D + threadIdx.x] = m;
                part[kRows * D + kRows + threadIdx.x] = l;
            }
            tc_fence_before();
        }
        if (!whole) {
            // An item that goes on in other CTAs: whoever arrives last joins the parts.
            const uint32_t f = share_of(sg.u0, total, workers), e = share_of(sg.u0 + sg.of - 1, total, workers);
            __threadfence();
            softmax_sync();
            if (threadIdx.x == 0) {
                sh.arrived = atomicAdd(p.counters + f, 1u) == e - f;
                if (sh.arrived)
                    p.counters[f] = 0;  // ready for the next call
            }
            softmax_sync();
            if (sh.arrived && r < rows) {
                __threadfence();
                auto at = [&](uint32_t i) { return p.parts + (2 * uint64_t(i) + (i == f ? 1 : 0)) * PF; };
                float mt = -INFINITY, lt = 0.f;
#pragma unroll 4
                for (uint32_t i = f; i <= e; i++)
                    mt = fmaxf(mt, __ldcg(at(i) + kRows * D + threadIdx.x));
                const float m0 = mt == -INFINITY ? 0.f : mt;
#pragma unroll 4
                for (uint32_t i = f; i <= e; i++)
                    lt = fmaf(exp2_fast(__ldcg(at(i) + kRows * D + threadIdx.x) - m0),
                              __ldcg(at(i) + kRows * D + kRows + threadIdx.x), lt);
#pragma unroll 1
                for (int d0 = 0; d0 < D; d0 += 32) {
                    float o[32];
#pragma unroll
                    for (int k = 0; k < 32; k++)
                        o[k] = 0.f;
#pragma unroll 2
                    for (uint32_t i = f; i <= e; i++) {
                        const float *const part = at(i);
                        float4 x[8];
#pragma unroll
                        for (int k = 0; k < 8; k++)
                            x[k] = __ldcg(reinterpret_cast<const float4 *>(part) + (d0 / 4 + k) * kRows + threadIdx.x);
                        const float w = exp2_fast(__ldcg(part + kRows * D + threadIdx.x) - m0);
#pragma unroll
                        for (int k = 0; k < 8; k++) {
                            o[4 * k] = fmaf(w, x[k].x, o[4 * k]);
                            o[4 * k + 1] = fmaf(w, x[k].y, o[4 * k + 1]);
                            o[4 * k + 2] = fmaf(w, x[k].z, o[4 * k + 2]);
                            o[4 * k + 3] = fmaf(w, x[k].w, o[4 * k + 3]);
                        }
                    }
                    store_dims<32>(p, sg.t0, sg.head, r, d0, o, mt, lt);
                }
            }
            softmax_sync();  // sh.arrived is read
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ PackedParams p) {
    using S = Sched<kRows, kKeys, kItemCost>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ Shared sh;
    // The row of units lies where the tiles will: it is not looked at after the first list is made.
    Row<kThreads> &row = *reinterpret_cast<Row<kThreads> *>(smem_raw);
    static_assert(sizeof(row) <= kSmem<D>, "");
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t raw = smem_addr(smem_raw), q_at = (raw + 1023u) & ~1023u;
    const uint32_t k_at = q_at + kQSlots * kTileBytes<D>, v_at = k_at + kStages * kTileBytes<D>;
    const uint32_t bars = smem_addr(sh.bars);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; i++) {
            const bool helpers = i < kQEmpty || (i >= kVOk && i < kVEmpty), rows = i >= kPFull && i < kPvDone,
                       both = (i >= kKEmpty && i < kVFull) || (i >= kVEmpty && i < kTurn);
            mbar_init(bars + 8 * i, helpers ? kHelper / 32 : rows ? 4 : both ? 2 : 1);
        }
        mbar_init_fence();
        sh.dead = 0;
    }
    grid_dep_launch();
    grid_dep_wait();
    const uint64_t total = build_row<S, kThreads, true>(p, row);
    const uint32_t workers = uint32_t(min((total + kMinShare - 1) / kMinShare, uint64_t(gridDim.x)));
    if (blockIdx.x >= workers)
        return;
    if (warp == kThreads / 32 - 1)
        tmem_alloc(smem_addr(&sh.tmem), kTmemCols);
    const uint64_t cut0 = mul_div(total, blockIdx.x, workers), cut1 = mul_div(total, blockIdx.x + 1, workers);
    // From here on every role walks through the lists of segments by itself;
    // barrier 0 stands before and after a list's work.  Registers a thread by
    // warpgroup: 2 x 184 + 88 + 56 = 4 x 128, the launch's.
    tc_fence_before();
    fence_proxy_async_smem();  // the row's memory is the copies' from then on
    if (warp < kSoftmax / 32) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        Item it{};
        if (warp == 0)
            it = locate<S>(p, row, cut0);
        uint32_t cnt = 0;
        for (uint64_t u = cut0; u < cut1;) {
            if (warp == 0) {
                int n;
                const uint64_t to = list_segments<S, kSegs>(p, it, u, cut1, sh.segs, &n);
                if (lane < n) {
                    sh.key0[lane] = __ldg(p.v.kstart + sh.segs[lane].s);
                    sh.hurt[lane] = 0;
                }
                if (lane == 0) {
                    sh.listed_to = to;
                    sh.n_segs = n;
                }
            }
            __syncthreads();
            tc_fence_after();
            u = sh.listed_to;
            softmax_role<D>(p, sh, bars, total, workers, cut0, cnt);
            __syncthreads();
        }
    } else if (warp < (kSoftmax + kHelper) / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        uint32_t steps = 0, halves = 0;
        for (uint64_t u = cut0; u < cut1;) {
            __syncthreads();
            u = sh.listed_to;
            helper_role<D>(p, sh, bars, q_at, v_at, steps, halves);
            __syncthreads();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        uint32_t steps = 0, halves = 0, cnt = 0, turns = 0;
        const int part = warp - (kSoftmax + kHelper) / 32;
        for (uint64_t u = cut0; u < cut1;) {
            __syncthreads();
            tc_fence_after();
            u = sh.listed_to;
            if (part < 2)
                mma_role<D>(p, sh, bars, q_at, k_at, v_at, part, steps, cnt, halves, turns);
            else if (part == 2 && elect_one())
                copy_role<D>(p, sh, bars, k_at, v_at, steps);
            __syncwarp();
            __syncthreads();
        }
    }
    if (warp == kThreads / 32 - 1)
        tmem_dealloc(sh.tmem, kTmemCols);
}

// K or V [n, heads, D] as boxes of 64 dimensions x 128 keys of one head; the dimensions in the order of
// their strides.
bool encode_keys_map(CUtensorMap *m, const Rows &r, int64_t n, int heads, int dim, bool *heads_outer, bool *one_head) {
    const auto enc = tensor_map_encoder();
    if (!enc)
        return false;
    *one_head = r.hs == 0;
    heads = *one_head ? 1 : heads;
    // (a dimension of one element has any stride)
    const int64_t hs = heads > 1 ? r.hs : dim, ts = n > 1 ? r.ts : std::max<int64_t>(hs * heads, dim);
    *heads_outer = hs > ts;
    const cuuint64_t of_heads = cuuint64_t(heads), of_keys = cuuint64_t(n);
    const cuuint64_t dims[3] = {cuuint64_t(dim), *heads_outer ? of_keys : of_heads, *heads_outer ? of_heads : of_keys};
    const cuuint64_t strides[2] = {cuuint64_t(std::min(hs, ts)) * 2, cuuint64_t(std::max(hs, ts)) * 2};
    const cuuint32_t box[3] = {64, *heads_outer ? cuuint32_t(kKeys) : 1u, *heads_outer ? 1u : cuuint32_t(kKeys)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Workspace: [error word | counters | parts].  The counters, which a call finds at zero, lie in
// the same place for every head size, so that one workspace serves all.
struct Layout {
    size_t counters, parts, total;
};
Layout layout(int head_dim) {
    const size_t ctas = size_t(sm_count());
    Layout w;
    w.counters = 256;
    w.parts = align_up(w.counters + 4 * ctas, 256);
    w.total = w.parts + 4 * 2 * ctas * kRows * (head_dim + 2);
    return w;
}

template <int D>
cudaError_t launch(const PackedParams &p, cudaStream_t st) {
    if (!ensure_smem(attention_kernel<D>, kSmem<D>))
        return cudaErrorUnknown;
    return launch_overlapped(attention_kernel<D>, dim3(unsigned(sm_count())), dim3(kThreads), kSmem<D>, st, p);
}

}  // namespace
}  // namespace uw

using namespace uw;

extern "C" uw_status uw_attention_workspace_size(int32_t head_dim, size_t *bytes) {
    if (!bytes)
        return UW_ERR_INVALID_ARG;
    if (head_dim <= 0)
        return UW_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128)
        return UW_ERR_UNSUPPORTED;
    *bytes = layout(head_dim).total;
    return UW_OK;
}

extern "C" uw_status uw_attention(const int32_t *start, const int32_t *kv_start, int32_t n_seqs, int64_t n_tokens,
                                  int64_t n_keys, const uw_kv4_rows *q, int32_t q_heads, const uw_kv4_rows *k,
                                  const uw_kv4_rows *v, int32_t kv_heads, int32_t head_dim, const uw_kv4_rows *out,
                                  float *lse, float softmax_scale, int32_t causal, int32_t window, void *ws,
                                  size_t ws_bytes, void *stream) {
    if (!q || !k || !v || !out || !ws || n_seqs < 0 || n_tokens < 0 || n_keys < 0 || window < 0 ||
        !std::isfinite(softmax_scale) || softmax_scale < 0.f || (reinterpret_cast<uintptr_t>(lse) & 3) ||
        ((reinterpret_cast<uintptr_t>(start) | reinterpret_cast<uintptr_t>(kv_start)) & 3) ||
        (reinterpret_cast<uintptr_t>(ws) & 255))
        return UW_ERR_INVALID_ARG;
    if (q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || head_dim <= 0)
        return UW_ERR_SHAPE;
    if (!kv_start && n_keys != n_tokens)
        return UW_ERR_SHAPE;
    PackedParams p{};
    p.c1 = (softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt(float(head_dim))) * 1.44269504089f;
    if ((head_dim != 64 && head_dim != 128) || q_heads > kKv4MaxHeads || n_tokens > 0x7fffffff || n_keys > 0x7fffffff ||
        n_tokens * (q_heads / kv_heads) > 0x7fffffff || !(p.c1 >= FLT_MIN) || !std::isfinite(p.c1))
        return UW_ERR_UNSUPPORTED;
    if (n_tokens == 0 || n_seqs == 0)
        return UW_OK;  // nothing to do needs no buffers (those of empty tensors are null)
    Rows keys{};
    if (!start || !kv4_rows(q, &p.q) || !kv4_rows(out, &p.o) ||
        (n_keys > 0 && (!kv4_rows(k, &keys) || !kv4_rows(v, &p.val))))
        return UW_ERR_INVALID_ARG;
    if (n_keys > 1 && (keys.ts == 0 || p.val.ts == 0))
        return UW_ERR_UNSUPPORTED;  // (copies need strides)
    const Layout w = layout(head_dim);
    if (ws_bytes < w.total)
        return UW_ERR_BUFFER_TOO_SMALL;
    uint8_t *const wsb = static_cast<uint8_t *>(ws);
    p.v = PackedView{start, kv_start ? kv_start : start, n_tokens, n_keys, n_seqs, kv_heads,
                     reinterpret_cast<uint32_t *>(wsb)};
    p.lse = lse;
    p.q_heads = q_heads;
    p.group = q_heads / kv_heads;
    p.by_group = Divisor(uint32_t(p.group));
    p.out32 = ((reinterpret_cast<uintptr_t>(p.o.p) | uintptr_t(p.o.ts) * 2 | uintptr_t(p.o.hs) * 2) & 31) == 0;
    p.causal = causal != 0;
    p.window = window;
    p.rows_min = 0;
    p.rows_max = INT32_MAX;
    p.counters = reinterpret_cast<uint32_t *>(wsb + w.counters);
    p.parts = reinterpret_cast<float *>(wsb + w.parts);
    // (without keys no tile is copied)
    if (n_keys > 0 && (!encode_keys_map(&p.kmap, keys, n_keys, kv_heads, head_dim, &p.heads_outer[0], &p.one_head[0]) ||
                       !encode_keys_map(&p.vmap, p.val, n_keys, kv_heads, head_dim, &p.heads_outer[1], &p.one_head[1])))
        return UW_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (head_dim == 128 ? launch<128>(p, st) : launch<64>(p, st)) == cudaSuccess ? UW_OK : UW_ERR_CUDA;
}
