// Attention over keys and values as they were projected (BF16 rows, no cache): whole
// sequences of different lengths behind each other, grouped heads.
//
// The floor is the tensor cores'.  One persistent CTA an SM takes an equal share of all
// (256 rows x 128 keys) steps (attn_work.cuh); a row is a query head of a token, rows of one
// kv head lie together, so a tile of K and V is read once for all of them.  Warp roles:
//   softmax   warps 0-3 and 4-7: the upper and lower 128 rows, a row a thread.  They read
//             S from tensor memory, take the exponentials and write P (BF16) over S, where
//             the second product reads it; at the end of an item they write the rows' output.
//   check     warps 8-11: V of tiles that some row does not see in full (see below);
//             queries where they do not come by a tensor map.
//   MMA       warps 12 and 13, for the upper and lower rows, one elected thread each: S = Q K^T and
//             O += P V with tcgen05.mma, 128 rows and 128 keys each.
//   copies    warp 14, one elected thread: tiles of K and V by tensor-map copies, two
//             stages of each.  V lies as it comes, [keys][dims], and is the second product's
//             operand with its rows along the product.
// A row's running maximum is only raised when its probabilities so far add up to
// more than 2^38 (BF16 and fp32 hold that without loss; with 2^24 a tile, which one row or another of a warp
// passes in every other tile, 8192 tokens, not causal, take 670 us instead of 593), so that after the first keys
// no score is compared and O is rarely rescaled.  P is rounded to one BF16 (2^-8, the one rounding beside
// the output's), as the product's operands have one type and V is BF16; what the rounding leaves, as a second operand, would be
// half as many products again.  Its sum is fp32 of the unrounded values, whose exponentials are off by about 2^-22.
//
// What a row does not see takes no part in it, whatever its bits: a masked score becomes -inf where it
// lies (an "open" tile, which not all rows see in full, takes 2200 cycles with that, 6000 with the mask in the
// loops of all else), and since 0 times a V that is not finite is not 0, the
// check warps look through V's tiles that are not seen by all rows, zero keys past the sequence's
// end and values that are not finite, and an item with such a value adds them at its end to the rows
// that see their keys.
//
// Measured, 32 query and 8 kv heads of 128, causal (cuBLAS's burst rate is 1919 TFLOP/s), from the best to the worst of
// several GPUs and clocks: 37 tokens 9.8 to 10.2 us, 2048 40.3 to 40.8 (843 to 853 TFLOP/s), 8192 318 to 326 (1690 to
// 1729), 16384 1206 to 1396 (1575 to 1823); 8192 not causal 593 to 660 (1667 to 1855); twelve packed prompts of 1 to
// 2000 tokens 62 to 64 (700); heads of 64, 8192 tokens 258 (1067), not causal 467 (1177); one token of each of 64 sequences over
// 4000 keys 171 (6.13 TB/s), 64 tokens over 16384 keys 53 (one row tile a head, cut into 19 shares).
// Long prompts are bound by the tensor cores (active in 75% of the cycles, not causal 81%, at
// the clock that the power leaves).  Short and packed ones pay for the share's begin (4 us until its first
// segment is listed, 3 more until Q, K and V of all CTAs are there), 3 us an item between its last products and
// the next one's first scores (output 2) and a join of parts (5.5).  With heads of 64 the
// products are half as long, and what bounds is the way from scores to probabilities and back through both
// halves (2085 cycles a step; tensor cores 39%, exponentials 39%).
// Outputs of items by the check warps instead, beside the next item's first tile: 21 prompts of 16 to 3001
// tokens 173 us instead of 164 (what runs seldom runs slowly: its instructions have to be fetched first).
// Exponentials by multiply-adds, one in eight: four sequences with heads of 64 124 us instead of 110.
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
// Of a kv head.  Rows are counted in 32 bits, past a sequence's last one up to the end of its tile.
constexpr int64_t kMostRows = 0x7fffffff - kRows;
constexpr int kSoftmax = 256, kCheck = 128;         // threads
constexpr int kThreads = kSoftmax + kCheck + 128;   // and a warpgroup of the MMA, copying and listing warps
// What an item costs beyond its steps, in steps (21 packed prompts 171 us, with 2 176, with 4 178).
constexpr int kItemCost = 3;
constexpr int kMinShare = 4;                          // units of a CTA at most, before more of them are used
constexpr int kSegs = 16;
constexpr int kStages = 2;
// 2^38: headroom of the sum of a row's probabilities.  A part's output stays below 2^38 |v|, the join of up to 152 of them
// below 2^46 |v|.
constexpr float kRaise = 274877906944.f;
constexpr uint32_t kTmemCols = 512;
// A call's number and a count of parts in one word: number * kCall + count.
constexpr uint64_t kCall = 1024;

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
    Divisor by_group, by_each;   // by_each.d: threads that look for the share's begin in one sequence (Plan)
    bool out32;                  // rows of o begin on 32-byte steps
    // of K and V: the tensor map's outermost dimension is the head; all heads are one
    bool heads_outer[2], one_head[2];
    bool q_map;                  // queries come by qmap
    int32_t rows_min, rows_max;  // any
    float *parts;                // parts of kRows * (D + 2) floats: output, maximum, sum
    unsigned long long *calls;     // kCall for each call there was
    unsigned long long *counters;  // [gridDim.x]: parts that are there of the item that begins in a CTA's share
    CUtensorMap kmap, vmap;      // 64 dimensions x 128 keys of one head
    CUtensorMap qmap;            // 64 dimensions x 128 rows: a kv head's query heads x tokens
};

enum Bar {
    kQFull, kQEmpty = kQFull + 2, kKFull = kQEmpty + 2, kKEmpty = kKFull + kStages, kVFull = kKEmpty + kStages,
    kVOk = kVFull + kStages, kVEmpty = kVOk + kStages, kTurn = kVEmpty + kStages, kSegFull = kTurn + 2,
    kSegFree = kSegFull + kSegs, kSFull = kSegFree + kSegs, kPFull = kSFull + 2, kPvDone = kPFull + 2,
    kDrain = kPvDone + 2, kJoin = kDrain + 2, kBars
};

struct Shared {
    uint64_t bars[kBars];
    Seg segs[kSegs];       // a ring: s < 0 after the last
    int32_t key0[kSegs];   // the sequence's first key
    uint32_t hurt[kSegs];  // V of a tile that not all rows see holds a value that is not finite
    uint64_t call;         // the call's number * kCall
    uint32_t tmem, dead, arrived;
};

template <int D>
constexpr uint32_t kTileBytes = kKeys * D * 2;  // 128 rows of Q, 128 keys of K or V
// With heads of 64 one warp issues all products (mma_role).
template <int D>
constexpr bool kOneMma = D == 64;
constexpr uint32_t kOutBytes = kSoftmax / 32 * 32 * 128;  // 64 dimensions of a softmax warp's rows
template <int D>
constexpr size_t kSmem = 1024 + kOutBytes + (2 + 2 * kStages) * size_t(kTileBytes<D>);

// Loops of what runs once an item or a tile are not unrolled: left to the compiler, this kernel had 310 KB of
// instructions instead of 139 (132 now), more than their caches hold (21 packed prompts 171 us instead of 164, a batch of
// five times 1000 tokens with heads of 64 73 instead of 62).
//
// A wait that every thread of a role makes at the same place.  One that runs
// out marks the kernel dead: all later waits return at once, every role
// walks through its remaining steps without waiting, and the status word tells.
__device__ __forceinline__ bool is_dead(Shared &sh) { return *reinterpret_cast<volatile uint32_t *>(&sh.dead) != 0; }
// What is ready, or soon, is found by a few looks; then a thread is suspended for up to a microsecond at a time
// (37 tokens 10.4 us, without the looks 11.4; long prompts the same).
constexpr uint32_t kHintNs = 1000;
__device__ __forceinline__ bool look(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity), "n"(kHintNs) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void wait(Shared &sh, uint32_t bar, uint32_t parity, uint32_t *status,
                                     uint32_t tries = kWaitTries) {
    for (int i = 0; i < 4; i++)
        if (look(bar, parity))
            return;
#pragma unroll 1
    for (uint32_t i = 0; i < tries; i++)
        if (try_wait(bar, parity) || is_dead(sh))
            return;
    atomicOr(status, kStatusTimeout);
    *reinterpret_cast<volatile uint32_t *>(&sh.dead) = 1;
}

// The same at a role's end, whatever became of the rest.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint32_t *status,
                                           uint32_t tries = kWaitTries) {
#pragma unroll 1
    for (uint32_t i = 0; i < tries; i++)
        if (try_wait(bar, parity))
            return;
    atomicOr(status, kStatusTimeout);
}

// Segment n of the CTA's share, once it is listed; null after the last.
__device__ __forceinline__ const Seg *segment(Shared &sh, uint32_t bars, uint32_t n, uint32_t *status) {
    wait(sh, bars + 8 * (kSegFull + n % kSegs), (n / kSegs) & 1, status);
    const Seg *const sg = sh.segs + n % kSegs;
    return is_dead(sh) || sg->s < 0 ? nullptr : sg;
}
// A warp (or the one thread of a role) is done with it.
template <int D>
constexpr uint32_t kSegUsers = (kSoftmax + kCheck) / 32 + (kOneMma<D> ? 2 : 3);
__device__ __forceinline__ void segment_done(uint32_t bars, uint32_t n) {
    mbar_arrive(bars + 8 * (kSegFree + n % kSegs));
}

// All softmax warps are here: a wait with a limit, as the halves may part where one has run out.
__device__ __forceinline__ void softmax_sync(Shared &sh, uint32_t bars, uint32_t &turns, uint32_t *status) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(bars + 8 * kJoin);
    wait(sh, bars + 8 * kJoin, turns++ & 1, status);
}

// Byte offset of 16-byte chunk c (8 values) of row r in a tile of 128 rows:
// blocks of 64 values, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    return uint32_t(c >> 3) * (128u * 128u) + sw128_offset(uint32_t(r), uint32_t(c & 7));
}

// The lowest n bits; none of n below 0, all of n past 32.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }

// Whether some row of the segment does not see some key of the tile at key0.
__device__ __forceinline__ bool is_open(const Seg &sg, int key0) {
    return key0 < sg.all_lo || sg.all_hi - key0 < kKeys;  // (key0 + kKeys may be 2^31)
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// All of the thread's groups of copies but the last are done.
__device__ __forceinline__ void cp_async_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}

// A value that is the same in all lanes, so that what follows from it stays in uniform
// registers, which the products' descriptors and addresses are taken from.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// The products of the upper rows (half 0) and the lower ones, or with kBoth of all.
//
// A step is a half's outputs of the last tile and, behind them, as S lies over P, its
// scores of the next; the halves in turns, so that one half's products run while the other's
// softmax does.  With heads of 128 a warp for each half takes turns with the other: an elected thread
// takes 60 cycles for each of 16 products and 140 for each wait, which for both halves is more than the
// tensor cores' 2048 (8192 tokens 324 us, by one warp 335; by two without turns, which interleave their
// products, 345, and twelve packed prompts 76 instead of 65).  With heads of 64 there are half as many products and
// one warp does (8192 tokens, not causal, 468 us, two 486).
template <int D, bool kBoth>
__device__ __forceinline__ void mma_role(const PackedParams &p, Shared &sh, uint32_t bars, uint32_t q_at,
                                         uint32_t k_at, uint32_t v_at, int part) {
    constexpr uint32_t kIdS = idesc_bf16_f32(128, kKeys), kIdO = idesc_bf16_f32(128, D) | kTransposeB;
    constexpr int kHalves = kBoth ? 2 : 1;
    const uint32_t tm = uint32_t(uniform(int(sh.tmem)));
    uint32_t steps = 0, turns = 0, cnt[kHalves] = {}, items[kHalves] = {};
    // Descriptors of the tiles; a step of 16 values along the first product adds 32
    // bytes, the next block of 64 values 128 * 128, a step of 16 keys along the second 16 * 128.
    const uint64_t q_desc = sdesc_sw128(q_at), k_desc = sdesc_sw128(k_at), v_desc = sdesc_sw128_n(v_at, 128 * 128);
    auto at = [](int i) { return uint64_t((i / 4) * (128 * 8) + (i % 4) * 2); };
#pragma unroll 1
    for (uint32_t n = 0;; n++) {
        const Seg *const sgp = segment(sh, bars, n, p.v.status);
        if (!uniform(sgp != nullptr))
            break;
        const Seg &sg = *sgp;
        const int tiles = uniform(sg.tiles), rows = uniform(sg.tokens * p.group - sg.rt * kRows);
        if (elect_one())
            segment_done(bars, n);
        __syncwarp();
        if (tiles == 0)
            continue;
        const bool two = rows > 128;
#pragma unroll 1
        for (int j = 0; j <= tiles; j++) {
            const uint32_t step = steps + j, before = step - 1, k_stage = step % kStages, v_stage = before % kStages;
            const uint64_t v = v_desc + v_stage * (kTileBytes<D> >> 4), k = k_desc + k_stage * (kTileBytes<D> >> 4);
            // (a wait takes 140 cycles, done or not: the one that all else waits for comes last)
            if (j < tiles)
                wait(sh, bars + 8 * (kKFull + k_stage), (step / kStages) & 1, p.v.status);
            if (j > 0)
                wait(sh, bars + 8 * (kVOk + v_stage), (before / kStages) & 1, p.v.status);
#pragma unroll
            for (int h = 0; h < kHalves; h++) {
                const int half = kBoth ? h : part;
                if (half && !two) {
                    if (!kBoth && elect_one()) {  // nothing to do with these tiles
                        if (j > 0)
                            mbar_arrive(bars + 8 * (kVEmpty + v_stage));
                        if (j < tiles)
                            mbar_arrive(bars + 8 * (kKEmpty + k_stage));
                    }
                    continue;
                }
                const uint32_t s_tm = tm + half * kKeys, o_tm = tm + 256 + half * D;
                if (j == 0)
                    wait(sh, bars + 8 * (kQFull + half), items[h]++ & 1, p.v.status);
                if (!kBoth && two)
                    wait(sh, bars + 8 * (kTurn + half), (turns++ & 1) ^ (half ^ 1), p.v.status);
                if (j > 0)
                    wait(sh, bars + 8 * (kPFull + half), cnt[h]++ & 1, p.v.status);
                tc_fence_after();
                if (elect_one()) {
                    if (j > 0) {
#pragma unroll
                        for (int i = 0; i < kKeys / 16; i++)
                            mma_ts(o_tm, s_tm + 8 * i, v + i * (16 * 8), kIdO, j > 1 || i > 0);
                        mma_commit(bars + 8 * (kPvDone + half));
                    }
                    if (j < tiles) {
                        const uint64_t q = q_desc + half * (kTileBytes<D> >> 4);
#pragma unroll
                        for (int i = 0; i < D / 16; i++)
                            mma_bf16(s_tm, q + at(i), k + at(i), kIdS, i > 0);
                        mma_commit(bars + 8 * (kSFull + half));
                        if (j == tiles - 1)
                            mma_commit(bars + 8 * (kQEmpty + half));
                    }
                    if (!kBoth || half == int(two)) {
                        if (j > 0)
                            mma_commit(bars + 8 * (kVEmpty + v_stage));
                        if (j < tiles)
                            mma_commit(bars + 8 * (kKEmpty + k_stage));
                    }
                    if (!kBoth && two)
                        mbar_arrive(bars + 8 * (kTurn + (half ^ 1)));
                }
                __syncwarp();
            }
        }
        steps += tiles;
    }
    // whatever became of the rest, all products are done before the barriers and the tensor memory go
    if (elect_one())
        mma_commit(bars + 8 * (kDrain + part));
    __syncwarp();
    drain_wait(bars + 8 * (kDrain + part), 0, p.v.status);
}

template <int D>
__device__ __forceinline__ void copy_role(const PackedParams &p, Shared &sh, uint32_t bars, uint32_t q_at,
                                          uint32_t k_at, uint32_t v_at) {
    uint32_t steps = 0, items[2] = {0, 0};
    auto copy_q = [&](int half, int kv_head, int token) {
        wait(sh, bars + 8 * (kQEmpty + half), (items[half] & 1) ^ 1, p.v.status);
        if (is_dead(sh))
            return;
        mbar_expect_tx(bars + 8 * (kQFull + half), kTileBytes<D>);
#pragma unroll
        for (int b = 0; b < D / 64; b++)
            tma_load_3d(q_at + half * kTileBytes<D> + b * (128 * 128), &p.qmap, 64 * b, kv_head * p.group, token,
                        bars + 8 * (kQFull + half));
        items[half]++;
    };
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
#pragma unroll 1
        for (int half = 0; half < 2; half++)
            if (items[half] > 0)
                drain_wait(bars + 8 * (kQFull + half), (items[half] - 1) & 1, p.v.status);
#pragma unroll 1
        for (uint32_t i = n - min(n, uint32_t(kStages)); i < n; i++) {
            drain_wait(bars + 8 * (kKFull + i % kStages), (i / kStages) & 1, p.v.status);
            if (i + less < n)
                drain_wait(bars + 8 * (kVFull + i % kStages), (i / kStages) & 1, p.v.status);
        }
    };
#pragma unroll 1
    for (uint32_t n = 0;; n++) {
        const Seg *const sgp = segment(sh, bars, n, p.v.status);
        if (!sgp)
            break;
        const int tiles = sgp->tiles, head = sgp->head, first = sh.key0[n % kSegs] + sgp->first * kKeys;
        // (with a map a half tile's 128 rows are whole tokens)
        const int rows = sgp->tokens * p.group - sgp->rt * kRows, token = sgp->t0 + p.by_group.of(sgp->rt * kRows);
        segment_done(bars, n);
        if (p.q_map && tiles > 0)
            copy_q(0, head, token);
#pragma unroll 1
        for (int j = 0; j < tiles; j++, steps++) {
            const uint32_t stage = steps % kStages, free = ((steps / kStages) & 1) ^ 1;
            const int key = first + j * kKeys;
            wait(sh, bars + 8 * (kKEmpty + stage), free, p.v.status);
            if (is_dead(sh))
                return drain(steps, 0);
            copy(p.kmap, 0, k_at + stage * kTileBytes<D>, head, key, bars + 8 * (kKFull + stage));
            if (p.q_map && j == 0 && rows > 128)
                copy_q(1, head, token + p.by_group.of(128));
            wait(sh, bars + 8 * (kVEmpty + stage), free, p.v.status);
            if (is_dead(sh))
                return drain(steps + 1, 1);
            copy(p.vmap, 1, v_at + stage * kTileBytes<D>, head, key, bars + 8 * (kVFull + stage));
        }
    }
    if (is_dead(sh))
        drain(steps, 0);
}

// Where row rr of a half of an item lies, chunk c.
__device__ __forceinline__ uint16_t *row_at(const PackedParams &p, const Rows &rows, const Seg &sg, int half, int rr,
                                            int c) {
    const int r = sg.rt * kRows + 128 * half + rr, i = p.by_group.of(r);
    return rows.p + (sg.t0 + int64_t(i)) * rows.ts + (sg.head * p.group + (r - i * p.group)) * rows.hs + 8 * c;
}
__device__ __forceinline__ int rows_of(const PackedParams &p, const Seg &sg, int half) {
    return min(sg.tokens * p.group - sg.rt * kRows - 128 * half, 128);
}

// V of tiles that some row does not see in full, and queries that do not come by a map.
template <int D>
__device__ __forceinline__ void check_role(const PackedParams &p, Shared &sh, uint32_t bars, uint32_t q_at,
                                           uint32_t v_at) {
    constexpr int C = D / 8;  // 16-byte chunks of a row
    const int t = threadIdx.x - kSoftmax, lane = t & 31;
    uint32_t steps = 0, items[2] = {0, 0};
    auto load_q = [&](const Seg *sgp) {
        if (p.q_map || !sgp || sgp->tiles == 0)
            return;
        const Seg &sg = *sgp;
        const int halves = rows_of(p, sg, 1) > 0 ? 2 : 1;
#pragma unroll 1
        for (int half = 0; half < halves; half++) {
            const int rows = rows_of(p, sg, half);
            wait(sh, bars + 8 * (kQEmpty + half), (items[half]++ & 1) ^ 1, p.v.status);
#pragma unroll 4
            for (int x = t; x < 128 * C; x += kCheck) {
                const int rr = x / C, c = x % C;
                const bool in = rr < rows;
                cp_async16_zfill(q_at + half * kTileBytes<D> + tile_at(rr, c),
                                 row_at(p, p.q, sg, half, in ? rr : 0, c), in ? 16 : 0);
            }
            cp_async_commit();
        }
#pragma unroll 1
        for (int half = 0; half < halves; half++) {
            if (half + 1 < halves)
                cp_async_wait_but_one();
            else
                cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bars + 8 * (kQFull + half));
        }
    };
    const Seg *sgp = segment(sh, bars, 0, p.v.status);
    load_q(sgp);
#pragma unroll 1
    for (uint32_t n = 0; sgp; n++) {
        const Seg &sg = *sgp;
#pragma unroll 1
        for (int j = 0; j < sg.tiles; j++, steps++) {
            const uint32_t stage = steps % kStages;
            const int key0 = (sg.first + j) * kKeys;
            wait(sh, bars + 8 * (kVFull + stage), (steps / kStages) & 1, p.v.status);
            if (is_open(sg, key0)) {
                // a key a thread
                const uint32_t tile = v_at + stage * kTileBytes<D>;
                const bool there = t < sg.len - key0;
                uint32_t any = 0;  // a sign bit for a value that is not finite
                if (there) {
#pragma unroll
                    for (int c = 0; c < C; c++) {
                        uint32_t w[4];
                        lds128(tile + tile_at(t, c), w);
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            any |= (w[k] & 0x7f807f80u) + 0x00800080u;
                    }
                }
                const bool hurt = (any & 0x80008000u) != 0;
                if (hurt || !there) {
#pragma unroll 1
                    for (int c = 0; c < C; c++) {
                        const uint32_t at = tile + tile_at(t, c);
                        uint32_t w[4];
                        lds128(at, w);
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const bool low = (w[k] & 0x7f80u) == 0x7f80u, high = (w[k] & 0x7f800000u) == 0x7f800000u;
                            w[k] = there ? w[k] & ((low ? 0u : 0xffffu) | (high ? 0u : 0xffff0000u)) : 0u;
                        }
                        sts128(at, w[0], w[1], w[2], w[3]);
                    }
                }
                if (hurt)
                    *reinterpret_cast<volatile uint32_t *>(&sh.hurt[n % kSegs]) = 1;
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bars + 8 * (kVOk + stage));
        }
        const Seg *const next = segment(sh, bars, n + 1, p.v.status);
        load_q(next);
        __syncwarp();
        if (lane == 0)
            segment_done(bars, n);
        sgp = next;
    }
}

// Where the CTA's share begins, found by all threads at once, of up to kThreads / 2 sequences: a thread stands for
// some row tiles of one sequence, their units (of one head) summed up over the threads.
struct Plan {
    uint64_t sums[kThreads / 32];
    uint64_t first[kThreads / 2 + 1];  // units of one head before each sequence
    uint64_t base, at;                 // the share's sequence and head: their first unit; its unit among one head's
    int32_t seq, head;
    Item item;
};
struct PlanThread {
    int32_t s, rt0;         // its sequence and first row tile
    Seq q;
    uint64_t before, mine;  // units of one head before its row tiles, and theirs
};
template <class S>
__device__ __forceinline__ uint64_t plan_units(const PackedParams &p, Plan &plan, PlanThread &me) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int each_seq = int(p.by_each.d), s = p.by_each.of(t), nth = t - s * each_seq;
    uint64_t n = 0;
    me.s = s;
    if (s < p.v.n_seqs) {
        const Seq q = seq_of(p.v, s);
        const int rts = S::mine(p, q) ? S::row_tiles(p, q) : 0, each = p.by_each.of(rts + each_seq - 1);
        const int rt0 = nth * each, rt1 = min(rt0 + each, rts);
        me.q = q;
        me.rt0 = rt0;
#pragma unroll 1
        for (int rt = rt0; rt < rt1; rt++)
            n += S::units(p, q, rt);
    }
    uint64_t upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o)
            upto += x;
    }
    if (lane == 31)
        plan.sums[warp] = upto;
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) {
        const uint64_t x = plan.sums[w];
        upto += w < warp ? x : 0;
        all += x;
    }
    if (s < p.v.n_seqs && nth == 0)
        plan.first[s] = upto - n;
    if (t == 0)
        plan.first[p.v.n_seqs] = all;
    __syncthreads();
    me.before = upto - n;
    me.mine = n;
    return all * p.v.heads;
}
// The item that holds unit u (of fewer than all) into plan.item; all threads call.
template <class S>
__device__ __forceinline__ void plan_item(const PackedParams &p, Plan &plan, uint64_t u, const PlanThread &me) {
    const int s = me.s;
    if (s < p.v.n_seqs && int(threadIdx.x) == s * int(p.by_each.d)) {
        const uint64_t lo = plan.first[s] * p.v.heads, per_head = plan.first[s + 1] - plan.first[s];
        if (u >= lo && u < lo + per_head * p.v.heads) {
            const uint64_t head = divide(u - lo, per_head);
            plan.seq = s;
            plan.head = int(head);
            plan.base = lo + head * per_head;
            plan.at = plan.first[s] + (u - plan.base);
        }
    }
    __syncthreads();
    if (s == plan.seq && plan.at >= me.before && plan.at - me.before < me.mine) {
        Item it;
        it.s = s;
        it.head = plan.head;
        it.q = me.q;
        uint64_t to = me.before;
#pragma unroll 1
        for (int rt = me.rt0;; rt++) {
            S::set_tile(p, it, rt);
            if (plan.at < to + it.n)
                break;
            to += it.n;
        }
        it.u0 = plan.base + (to - plan.first[s]);
        plan.item = it;
    }
}

// The segments of the CTA's share from unit u (in item `it`) on, one after the other into the ring; a warp.
template <class S>
__device__ __forceinline__ void list_role(const PackedParams &p, Shared &sh, uint32_t bars, Item &it, uint64_t u,
                                          uint64_t end) {
#pragma unroll 1
    for (uint32_t n = 0;;) {
        const uint32_t slot = n % kSegs;
        wait(sh, bars + 8 * (kSegFree + slot), ((n / kSegs) & 1) ^ 1, p.v.status);
        if (is_dead(sh))
            break;
        int found = 0;
        if (u < end)
            u = list_segments<S, 1>(p, it, u, end, sh.segs + slot, &found);
        if (found == 0 && u < end)
            continue;
        if ((threadIdx.x & 31) == 0) {
            if (found) {
                sh.key0[slot] = __ldg(p.v.kstart + sh.segs[slot].s);
                sh.hurt[slot] = 0;
            } else {
                sh.segs[slot].s = -1;
            }
            mbar_arrive(bars + 8 * (kSegFull + slot));
        }
        if (!found)
            break;
        n++;
    }
}

template <int D>
__device__ __forceinline__ void softmax_role(const PackedParams &p, Shared &sh, uint32_t bars, uint64_t total,
                                             uint32_t workers, uint64_t cut0, uint32_t out_at) {
    constexpr int PF = kRows * (D + 2);
    const int half = threadIdx.x >> 7, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t s_tm = sh.tmem + lanes + half * kKeys, o_tm = sh.tmem + lanes + 256 + half * D;
    const uint64_t c1 = pair2(p.c1, p.c1);
    uint32_t cnt = 0, turns = 0;
#pragma unroll 1
    for (uint32_t n = 0;; n++) {
        const Seg *const sgp = segment(sh, bars, n, p.v.status);
        if (!sgp)
            break;
        const Seg &sg = *sgp;
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
        // The maximum; the sum of probabilities from which it is raised (any, as long as there is
        // none; never where there will be none).
        const float unset = mine.hi > mine.lo ? -1.f : INFINITY;
        float m = -INFINITY, lim = unset, room = unset;  // room: what of lim is left for a tile
        uint64_t mm = 0, l2 = 0;          // less the maximum, and the sum, in pairs
#pragma unroll 1
        for (int j = 0; active && j < sg.tiles; j++) {
            const int key0 = (sg.first + j) * kKeys;
            wait(sh, bars + 8 * (kSFull + half), cnt & 1, p.v.status);
            tc_fence_after();
            // The first scores, before it is known what the tile needs (16 heads of 64, 8192 tokens, not
            // causal, 253 us, loaded after that 260).
            uint32_t x[2][32];
            tmem_ld32(s_tm, x[0]);
            const int lo = mine.lo - key0, hi = mine.hi - key0;  // the row's keys of the tile
            const bool open = is_open(sg, key0);
            bool over = j == 0, last = open && j == 0;  // the row's maximum is to be raised; it is that of all keys
            int look = open ? kKeys : j == 0 ? 32 : 0;  // the scores to be looked at first
            tmem_ld_wait();
#pragma unroll 1
            for (;; last = true, look = kKeys) {
                if (look > 0) {
                    // What the row does not see becomes -inf, whose exponential is 0; from there on an open tile is
                    // like others.  And the highest score of the first 32 keys (of an item's first tile, where all
                    // see it: most often that will do) or of all.
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < look; c += 32) {
                        uint32_t x[32];
                        tmem_ld32(s_tm + c, x);
                        tmem_ld_wait();
                        const uint32_t seen = bits_below(hi - c) & ~bits_below(lo - c);
                        if (__any_sync(0xffffffffu, seen != 0xffffffffu)) {
#pragma unroll
                            for (int k = 0; k < 32; k++)
                                x[k] = seen >> k & 1 ? x[k] : 0xff800000u;
                            tmem_st32(s_tm + c, x);
                        }
#pragma unroll
                        for (int k = 0; k < 32; k++)
                            top = fmaxf(top, __uint_as_float(x[k]));
                    }
                    tmem_st_wait();
                    if (__any_sync(0xffffffffu, over)) {
                        // Raised in rows that need it by their own sum: what the row has so far is scaled down.
                        // By the sum's logarithm at least, so that it is 1 at most whatever this tile's scores are.
                        const float2 lf = unpair(l2);
                        const float m2 = over ? fmaxf(fmaxf(m, m + __log2f(lf.x + lf.y)), top * p.c1) : m;
                        const float m20 = m2 == -INFINITY ? 0.f : m2;
                        const float f = !over ? 1.f : m == -INFINITY ? 0.f : exp2_fast(m - m20);
                        l2 = mul2(l2, pair2(f, f));
                        m = m2;
                        mm = pair2(-m20, -m20);
                        lim = room = m2 == -INFINITY ? unset : kRaise;
                        if (j > 0) {
                            wait(sh, bars + 8 * (kPvDone + half), (cnt - 1) & 1, p.v.status);
                            tc_fence_after();
#pragma unroll 1
                            for (int d0 = 0; d0 < D; d0 += 16) {
                                uint32_t w[16];
                                tmem_ld16(o_tm + d0, w);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 16; i++)
                                    w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
                                tmem_st16(o_tm + d0, w);
                            }
                        }
                    }
                    tmem_ld32(s_tm, x[0]);
                    tmem_ld_wait();
                }
                // Scores are loaded 32 ahead of those whose exponentials are taken.
                uint32_t pk[2][32];
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    if (c > 0)
                        tmem_ld_wait();
                    if (c < 3)
                        tmem_ld32(s_tm + 32 * (c + 1), x[(c + 1) & 1]);
#pragma unroll
                    for (int k = 0; k < 16; k++) {
                        const uint32_t *const w = x[c & 1] + 2 * k;
                        const float2 y = unpair(fma2(pair2(__uint_as_float(w[0]), __uint_as_float(w[1])), c1, mm));
                        const float a = exp2_fast(y.x), b = exp2_fast(y.y);
                        sum[k & 1] = add2(sum[k & 1], pair2(a, b));
                        pk[c >> 1][16 * (c & 1) + k] = bf16_pack(a, b);
                    }
                }
                sum[0] = add2(sum[0], sum[1]);
                const float2 f = unpair(sum[0]);
                over = f.x + f.y > room;
                if (!last && __any_sync(0xffffffffu, over))
                    continue;
                l2 = add2(l2, sum[0]);
                tmem_st32(s_tm, pk[0]);
                tmem_st32(s_tm + 32, pk[1]);
                break;
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bars + 8 * (kPFull + half));
            cnt++;
            // (here, where nothing waits for it: before the comparison 163 us for 21 packed prompts instead of 160)
            const float2 lf = unpair(l2);
            room = lim - (lf.x + lf.y);
        }

        const float2 lf = unpair(l2);
        const float l = lf.x + lf.y;
        const bool whole = sg.tiles == sg.of, valued = active && sg.tiles > 0;
        const int slot = cut0 > sg.u0 ? 0 : 1;
        float *const part = p.parts + (2 * uint64_t(blockIdx.x) + slot) * PF;
        // An item that goes on in other CTAs: whoever comes last joins the parts.  If all others are there already (as
        // they are where the item begins at the end of a share), this part needs not go through memory (2048 tokens
        // 41.0 us, otherwise 43.7).
        uint32_t f = 0, e = 0;
        bool last = false;
        if (!whole) {
            f = share_of(sg.u0, total, workers);
            e = share_of(sg.u0 + sg.of - 1, total, workers);
            if (threadIdx.x == 0)
                sh.arrived = *reinterpret_cast<volatile unsigned long long *>(p.counters + f) == sh.call + (e - f);
            softmax_sync(sh, bars, turns, p.v.status);
            last = sh.arrived;
        }
        if (valued) {
            wait(sh, bars + 8 * (kPvDone + half), (cnt - 1) & 1, p.v.status);
            tc_fence_after();
        }
        const bool hurt = valued && *reinterpret_cast<volatile uint32_t *>(&sh.hurt[n % kSegs]) != 0;
        if (hurt) {
            // values of V that are not finite, of the keys that the row sees in tiles that not all do
            const int last = min(mine.hi - 1, (sg.first + sg.tiles - 1) * kKeys + (kKeys - 1));
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {
                uint32_t w[32];
                tmem_ld32(o_tm + d0, w);
                tmem_ld_wait();
#pragma unroll 1
                for (int key = max(mine.lo, sg.first * kKeys); key <= last; key++) {
                    if (!is_open(sg, key & ~(kKeys - 1)))
                        continue;
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        p.val.p + (sh.key0[n % kSegs] + int64_t(key)) * p.val.ts + sg.head * p.val.hs + d0);
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        const uint4 v = __ldg(src + c);
                        const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            uint32_t &low = w[8 * c + 2 * i], &high = w[8 * c + 2 * i + 1];
                            if ((a[i] & 0x7f80u) == 0x7f80u)
                                low = __float_as_uint(__uint_as_float(low) + bf16_lo(a[i]));
                            if ((a[i] & 0x7f800000u) == 0x7f800000u)
                                high = __float_as_uint(__uint_as_float(high) + bf16_hi(a[i]));
                        }
                    }
                }
                __syncwarp();
                tmem_st32(o_tm + d0, w);
            }
            tmem_st_wait();
        }
        if (active && !last) {
            const float inv = l == 0.f ? 0.f : 1.f / l;  // no key: o is 0 and stays 0
            // A warp's rows lie in shared memory for a moment, 64 dimensions at a time, so that they go out by whole
            // lines (8192 tokens 324 us, stored by rows of their threads 340).
            const uint32_t mine_at = out_at + warp * (32 * 128);
            const int in_half = min(int(threadIdx.x & 127), rows - r0 - 128 * half - 1);
            const uint64_t row_of = reinterpret_cast<uint64_t>(row_at(p, p.o, sg, half, in_half, 0));
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {
                uint32_t w[32];
                if (valued) {
                    tmem_ld32(o_tm + d0, w);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        w[i] = 0;
                }
                auto o = [&](int i) { return __uint_as_float(w[i]); };
                if (!whole) {
                    if (r < rows) {
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            reinterpret_cast<float4 *>(part)[(d0 / 4 + i) * kRows + threadIdx.x] =
                                make_float4(o(4 * i), o(4 * i + 1), o(4 * i + 2), o(4 * i + 3));
                    }
                    continue;
                }
#pragma unroll
                for (int c = 0; c < 4; c++)
                    sts128(mine_at + sw128_offset(lane, (d0 & 63) / 8 + c),
                           bf16_pack(o(8 * c) * inv, o(8 * c + 1) * inv),
                           bf16_pack(o(8 * c + 2) * inv, o(8 * c + 3) * inv),
                           bf16_pack(o(8 * c + 4) * inv, o(8 * c + 5) * inv),
                           bf16_pack(o(8 * c + 6) * inv, o(8 * c + 7) * inv));
                if ((d0 & 63) != 32)
                    continue;
                __syncwarp();
#pragma unroll 4
                for (int k = 0; k < 8; k++) {
                    const int row = 4 * k + (lane >> 3), c = lane & 7;
                    const uint64_t to = __shfl_sync(0xffffffffu, row_of, row) + 2 * (d0 - 32) + 16 * c;
                    uint32_t v[4];
                    lds128(mine_at + sw128_offset(row, c), v);
                    if (r0 + 32 * warp + row < rows)
                        *reinterpret_cast<uint4 *>(to) = make_uint4(v[0], v[1], v[2], v[3]);
                }
                __syncwarp();
            }
            tc_fence_before();
            if (!whole) {
                part[kRows * D + threadIdx.x] = m;
                part[kRows * D + kRows + threadIdx.x] = l;
            } else if (p.lse && r < rows) {
                const int i = p.by_group.of(r);
                p.lse[(sg.t0 + int64_t(i)) * p.q_heads + sg.head * p.group + (r - i * p.group)] =
                    l == 0.f ? -INFINITY : 0.69314718056f * (m + log2f(l));
            }
        }
        if (!whole) {
            if (!last) {
                __threadfence();
                softmax_sync(sh, bars, turns, p.v.status);
                if (threadIdx.x == 0) {
                    atomicMax(p.counters + f, sh.call);  // what an earlier call left is less
                    sh.arrived = atomicAdd(p.counters + f, 1ull) == sh.call + (e - f);
                }
                softmax_sync(sh, bars, turns, p.v.status);
                last = sh.arrived;
            }
            if (last && active) {
                __threadfence();
                auto at = [&](uint32_t i) { return p.parts + (2 * uint64_t(i) + (i == f ? 1 : 0)) * PF; };
                float mt = -INFINITY, lt = 0.f;
#pragma unroll 2
                for (uint32_t i = f; i <= e; i++) {
                    const bool own = i == blockIdx.x;
                    const float mi = own ? m : __ldcg(at(i) + kRows * D + threadIdx.x);
                    const float li = own ? l : __ldcg(at(i) + kRows * D + kRows + threadIdx.x);
                    const float m2 = fmaxf(mt, mi), m20 = m2 == -INFINITY ? 0.f : m2;
                    lt = fmaf(exp2_fast(mi - m20), li, lt * exp2_fast(mt - m20));
                    mt = m2;
                }
                const float m0 = mt == -INFINITY ? 0.f : mt;
#pragma unroll 1
                for (int d0 = 0; d0 < D; d0 += 64) {
                    float o[64];
#pragma unroll
                    for (int k = 0; k < 64; k++)
                        o[k] = 0.f;
#pragma unroll 1
                    for (uint32_t i = f; i <= e; i++) {
                        const float *const from = at(i);
                        float x[64];
                        const bool own = i == blockIdx.x;
                        if (own) {  // still there
                            uint32_t w[2][32];
                            tmem_ld32(o_tm + d0, w[0]);
                            tmem_ld32(o_tm + d0 + 32, w[1]);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 64; k++)
                                x[k] = __uint_as_float(w[k / 32][k % 32]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 16; k++)
                                *reinterpret_cast<float4 *>(x + 4 * k) = __ldcg(
                                    reinterpret_cast<const float4 *>(from) + (d0 / 4 + k) * kRows + threadIdx.x);
                        }
                        const float w = exp2_fast((own ? m : __ldcg(from + kRows * D + threadIdx.x)) - m0);
#pragma unroll
                        for (int k = 0; k < 64; k++)
                            o[k] = fmaf(w, x[k], o[k]);
                    }
                    if (r < rows)
                        store_dims<64>(p, sg.t0, sg.head, r, d0, o, mt, lt);
                }
                tc_fence_before();
            }
            softmax_sync(sh, bars, turns, p.v.status);  // sh.arrived is read
        }
        __syncwarp();
        if (lane == 0)
            segment_done(bars, n);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ PackedParams p) {
    using S = Sched<kRows, kKeys, kItemCost>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ Shared sh;
    // What the share's begin is found with lies where the tiles will: it is not looked at after the first segment is
    // listed.
    Row<kThreads> &row = *reinterpret_cast<Row<kThreads> *>(smem_raw);
    Plan &plan = *reinterpret_cast<Plan *>(smem_raw);
    static_assert(sizeof(row) <= kSmem<D> && sizeof(plan) <= kSmem<D>, "");
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
    const uint32_t raw = smem_addr(smem_raw), q_at = (raw + 1023u) & ~1023u;
    const uint32_t out_at = q_at + 2 * kTileBytes<D>, k_at = out_at + kOutBytes;
    const uint32_t v_at = k_at + kStages * kTileBytes<D>;
    const uint32_t bars = smem_addr(sh.bars);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; i++) {
            uint32_t n = 1;  // a commit, a copy's announcement
            if ((i < kQEmpty && !p.q_map) || (i >= kVOk && i < kVEmpty))
                n = kCheck / 32;
            else if (i >= kPFull && i < kPvDone)
                n = 4;
            else if ((i >= kKEmpty && i < kVFull) || (i >= kVEmpty && i < kTurn))
                n = kOneMma<D> ? 1 : 2;
            else if (i >= kSegFree && i < kSFull)
                n = kSegUsers<D>;
            else if (i == kJoin)
                n = kSoftmax / 32;
            mbar_init(bars + 8 * i, n);
        }
        mbar_init_fence();
        sh.dead = 0;
        prefetch_map(&p.kmap);
        prefetch_map(&p.vmap);
        prefetch_map(&p.qmap);
    }
    grid_dep_launch();
    grid_dep_wait();
    // The call's number.  All CTAs' additions are kCall, and each makes its own as it reads, so that the first digits
    // are the same for all of them.
    unsigned long long call = 0;
    if (threadIdx.x == 0)
        call = atomicAdd(p.calls, blockIdx.x == 0 ? kCall + 1 - gridDim.x : 1ull);
    const bool few = p.v.n_seqs <= kThreads / 2;
    PlanThread me{};
    const uint64_t total = few ? plan_units<S>(p, plan, me) : build_row<S, kThreads, true>(p, row);
    const uint32_t workers = uint32_t(min((total + kMinShare - 1) / kMinShare, uint64_t(gridDim.x)));
    if (blockIdx.x >= workers)
        return;
    if (warp == kThreads / 32 - 1)
        tmem_alloc(smem_addr(&sh.tmem), kTmemCols);
    const uint64_t cut0 = mul_div(total, blockIdx.x, workers), cut1 = mul_div(total, blockIdx.x + 1, workers);
    if (few) {
        plan_item<S>(p, plan, cut0, me);
        __syncthreads();
    }
    Item it{};
    if (warp == kThreads / 32 - 1)
        it = few ? plan.item : locate<S>(p, row, cut0);
    if (threadIdx.x == 0)
        sh.call = call / kCall * kCall;
    tc_fence_before();
    fence_proxy_async_smem();  // the row's memory is the copies' from here on
    __syncthreads();
    tc_fence_after();
    // From here on every role walks through the segments by itself.  Registers a thread by
    // warpgroup: 2 x 176 + 88 + 72 = 4 x 128, the launch's.
    if (warp < kSoftmax / 32) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        softmax_role<D>(p, sh, bars, total, workers, cut0, out_at);
    } else if (warp < (kSoftmax + kCheck) / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        check_role<D>(p, sh, bars, q_at, v_at);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int part = warp - (kSoftmax + kCheck) / 32;
        if (part == 0 || (part == 1 && !kOneMma<D>)) {
            mma_role<D, kOneMma<D>>(p, sh, bars, q_at, k_at, v_at, part);
        } else if (part == 2) {
            if (elect_one())
                copy_role<D>(p, sh, bars, q_at, k_at, v_at);
        } else if (part == 3) {
            list_role<S>(p, sh, bars, it, cut0, cut1);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kThreads / 32 - 1)
        tmem_dealloc(sh.tmem, kTmemCols);
}

// Waits that nothing ends, by one thread: the first gives up, says so and marks the kernel dead; one after it returns
// at once and says nothing; a drain gives up and says so.  The status word holds a timeout only if all three did.
__global__ void withheld_arrival_kernel(uint32_t *status, uint32_t tries) {
    __shared__ Shared sh;
    const uint32_t bar = smem_addr(sh.bars);
    mbar_init(bar, 1);
    mbar_init_fence();
    sh.dead = 0;
    wait(sh, bar, 0, status, tries);
    if (!(atomicExch(status, 0u) & kStatusTimeout) || !is_dead(sh))
        return;
    wait(sh, bar, 0, status);
    if (atomicExch(status, 0u) == 0)
        drain_wait(bar, 0, status, tries);
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

// Q as boxes of 64 dimensions x a kv head's query heads x the tokens of 128 rows, where that comes out even and
// rows lie in that order; otherwise the kernel does without.
bool encode_q_map(CUtensorMap *m, const Rows &r, int64_t n, int heads, int dim, int group) {
    const auto enc = tensor_map_encoder();
    const int64_t hs = heads > 1 ? r.hs : dim, ts = n > 1 ? r.ts : std::max<int64_t>(hs * heads, dim);
    if (!enc || group > 128 || 128 % group || hs == 0 || ts < hs)
        return false;
    const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(n)};
    const cuuint64_t strides[2] = {cuuint64_t(hs) * 2, cuuint64_t(ts) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(group), cuuint32_t(128 / group)}, estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Workspace: [error word | calls there were | counters | parts].  Calls and counters lie in the same place for every head
// size, so that one workspace serves all.  A counter's word holds its call's number too: parts of an item that never came to
// their end, as the call ran out of time, count for no later one.
struct Layout {
    size_t calls, counters, parts, total;
};
Layout layout(int head_dim) {
    const size_t ctas = size_t(sm_count());
    Layout w;
    w.calls = 256;
    w.counters = w.calls + 8;
    w.parts = align_up(w.counters + 8 * ctas, 256);
    w.total = w.parts + 4 * 2 * ctas * kRows * (head_dim + 2);
    return w;
}

template <int D>
cudaError_t launch(const PackedParams &p, cudaStream_t st) {
    if (sm_count() >= int(kCall) || !ensure_smem(attention_kernel<D>, kSmem<D>))
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
        n_tokens * (q_heads / kv_heads) > kMostRows || !(p.c1 >= FLT_MIN) || !std::isfinite(p.c1))
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
    p.by_each = Divisor(uint32_t(std::max(kThreads / n_seqs, 1)));
    p.out32 = ((reinterpret_cast<uintptr_t>(p.o.p) | uintptr_t(p.o.ts) * 2 | uintptr_t(p.o.hs) * 2) & 31) == 0;
    p.causal = causal != 0;
    p.window = window;
    p.rows_min = 0;
    p.rows_max = INT32_MAX;
    p.calls = reinterpret_cast<unsigned long long *>(wsb + w.calls);
    p.counters = reinterpret_cast<unsigned long long *>(wsb + w.counters);
    p.parts = reinterpret_cast<float *>(wsb + w.parts);
    // (without keys no tile is copied)
    if (n_keys > 0 && (!encode_keys_map(&p.kmap, keys, n_keys, kv_heads, head_dim, &p.heads_outer[0], &p.one_head[0]) ||
                       !encode_keys_map(&p.vmap, p.val, n_keys, kv_heads, head_dim, &p.heads_outer[1], &p.one_head[1])))
        return UW_ERR_CUDA;
    p.q_map = encode_q_map(&p.qmap, p.q, n_tokens, q_heads, head_dim, p.group);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (head_dim == 128 ? launch<128>(p, st) : launch<64>(p, st)) == cudaSuccess ? UW_OK : UW_ERR_CUDA;
}

extern "C" uw_status uw_selftest_attention_wait(void *ws, size_t ws_bytes, uint32_t tries, void *stream) {
    if (!ws || tries == 0 || tries > kWaitTries)
        return UW_ERR_INVALID_ARG;
    if (ws_bytes < 256)
        return UW_ERR_BUFFER_TOO_SMALL;
    withheld_arrival_kernel<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<uint32_t *>(ws), tries);
    return cudaGetLastError() == cudaSuccess ? UW_OK : UW_ERR_CUDA;
}
