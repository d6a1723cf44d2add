// Attention over the 4-bit paged cache for sequences with many rows (new
// tokens x query heads of a kv head): prompts and their chunks.
//
// The floor is the tensor cores'; what bounds the kernel is the chain of each
// softmax warp from a score to its probability: a step (256 rows x 128 keys) of
// 4860 cycles has the tensor cores busy for 38%, the exponential unit for 19%,
// the fp32 units for 36% and issue slots for 46%, and two softmax warps a
// scheduler are what registers and tensor memory (256 columns of scores, 256 of
// outputs) allow.  So every key of an item is unpacked once for 256 rows, and a
// softmax thread has as many independent scores in flight as its registers hold.
// One persistent CTA an SM takes an equal share of all (256 rows x 128 keys)
// steps (kv4_attn.cuh).  Warp roles:
//   softmax   warps 0-3 and 4-7: the upper and lower 128 rows, 32 a warp.  They
//             read S from tensor memory, apply the keys' scales and offsets and
//             the mask, take the exponentials and write P s (BF16) over S, where
//             the second product reads it; at the end of an item they write
//             the rows' output.
//   unpack    warps 8-11: codes from global memory (loaded a tile ahead) to BF16
//             tiles in shared memory, K as [keys][dims], V transposed as
//             [dims][keys], both K-major for the tensor cores; the scales and
//             offsets; the queries of an item.
//   MMA       warp 12, one elected thread (the rest of the warp walks along, which
//             keeps descriptors and addresses in uniform registers): S = Q K^T and O += (P s) V with
//             tcgen05.mma, 128 rows and half a step's keys each: while the softmax
//             works on one half of the keys, the products of the other half run.
// Both products take the codes as they are (Codes in kv4_codes.cuh: integers in units
// of 2^-133, no rounded K or V), the queries and probabilities scaled up
// against them.  The running maximum is only raised when some thread's sixteen
// probabilities of a row and 64 keys add up to more than 2^24 (BF16 and fp32 hold
// that without loss), so that no score is compared and O is rarely rescaled.
// P s is rounded to one BF16 (the sum of the values' middles is fp32): its rest
// as a second operand, as the kernel for few rows has it, would cost the softmax
// warps, which bound this one, a difference, a packing and a store for each score.
// Prompts are 0.0022 off from 64 bits in the 2-norm, with 0.0017 the output's
// own rounding.
//
// Measured, 32 query and 8 kv heads of 128, causal:
//   a prompt of 8192 tokens                 654 us (841 TFLOP/s, 0.44 of cuBLAS's burst)
//   64 new tokens after 524288              605 us (908 TFLOP/s)
//   a prompt of 2048 tokens                 81 us (427 TFLOP/s): to the first scores 9 us, an item's
//                                           output 2, a join 3 to 8
// Tried beside this: 32 keys at a time with the next scores on their way 778 us
// (less to do at a time for each warp), no branch between scores and P 700,
// the two halves' exponentials in turns 689, one half started later 677.
#include <cmath>
#include <type_traits>

#include "kernels.h"
#include "kv4_attn.cuh"
#include "kv4_codes.cuh"
#include "tmem.cuh"

namespace uw {

namespace {

constexpr int kRows = 256, kKeys = 128;
constexpr int kSoftmax = 256, kUnpack = 128;          // threads
constexpr int kThreads = kSoftmax + kUnpack + 128;    // and a warpgroup whose first warp issues the products
// What an item costs beyond its steps, in steps (a prompt of 8192 tokens: 675 us, with 0 847).
constexpr int kItemCost = 3;
// Units of a CTA at least: an item in many parts is joined part after part (128
// tokens of 8 heads after 8000 keys 55 us, with one unit 84; other short calls alike).
constexpr int kMinShare = 4;
constexpr int kSegs = 32;
constexpr int kStages = 2, kParStages = 4;
constexpr float kRaise = 16777216.f;                  // 2^24: headroom of a thread's 16 probabilities of 64 keys
constexpr uint32_t kTmemCols = 512;

enum Bar {
    kQFull, kQEmpty, kKFull, kKEmpty = kKFull + kStages, kVFull = kKEmpty + kStages, kVEmpty = kVFull + kStages,
    kParFull = kVEmpty + kStages,
    kSFull = kParFull + kParStages, kPFull = kSFull + 4,  // [rows' half][keys' half]
    kPvDone = kPFull + 4, kBars = kPvDone + 4
};

struct Shared {
    uint64_t bars[kBars];
    uint64_t listed_to;
    Seg segs[kSegs];
    float qs[2][kRows];                    // sums of the queries, of this item and the next
    float4 kpar[kParStages][kKeys / 2];    // (a, a', b, b') of two keys: y = a (q.c) + b sum q
    float4 vpar[kParStages][kKeys / 2];    // (s, s', mid, mid')
    Row<kThreads> row;
    uint32_t tmem, dead, arrived;
    int n_segs;
};

template <int D>
constexpr uint32_t kTileBytes = kKeys * D * 2;  // 128 rows of Q, 128 keys of K, D dimensions of V
template <int D>
constexpr size_t kSmem = 1024 + (2 + 2 * kStages) * size_t(kTileBytes<D>);

// A wait that every thread of a role makes at the same place.  One that runs
// out marks the kernel dead: all later waits return at once, every role
// walks through its remaining steps without waiting, and the status word tells.
__device__ __forceinline__ void wait(Shared &sh, uint32_t bar, uint32_t parity, uint32_t *status) {
    if (mbar_try_wait(bar, parity) || *reinterpret_cast<volatile uint32_t *>(&sh.dead))
        return;
    if (!mbar_wait(bar, parity, status, kStatusTimeout))
        *reinterpret_cast<volatile uint32_t *>(&sh.dead) = 1;
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Byte offset of 16-byte chunk c (8 values) of row r in a tile of `rows` rows:
// blocks of 64 values, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(int r, int c, int rows) {
    return uint32_t(c >> 3) * uint32_t(rows) * 128u + sw128_offset(uint32_t(r), uint32_t(c & 7));
}

template <int D>
__device__ __forceinline__ void mma_role(const AttnParams &p, Shared &sh, uint32_t bars, uint32_t q_at, uint32_t k_at,
                                         uint32_t v_at, uint32_t &steps, uint32_t (&cnt)[2], uint32_t &items) {
    constexpr uint32_t kIdS = idesc_bf16_f32(128, kKeys / 2), kIdO = idesc_bf16_f32(128, D);
    const uint32_t tm = sh.tmem;
    // Descriptors of the tiles; a step of 16 values along the product adds 32
    // bytes, the next block of 64 values `rows` * 128 (both in units of 16 bytes).
    const uint64_t q_desc = sdesc_sw128(q_at), k_desc = sdesc_sw128(k_at), v_desc = sdesc_sw128(v_at);
    auto at = [](int i, int rows) { return uint64_t((i / 4) * (rows * 8) + (i % 4) * 2); };
    // Scores of 128 rows and half a step's keys, and the output of the same.
    auto score = [&](int half, uint32_t step, int h) {
        const uint64_t q = q_desc + half * (kTileBytes<D> >> 4);
        const uint64_t k = k_desc + (step % kStages) * (kTileBytes<D> >> 4) + h * (kKeys / 2 * 8);
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < D / 16; i++)
                mma_bf16(tm + half * kKeys + h * (kKeys / 2), q + at(i, 128), k + at(i, kKeys), kIdS, i > 0);
            mma_commit(bars + 8 * (kSFull + 2 * half + h));
        }
        __syncwarp();
    };
    auto output = [&](int half, uint32_t step, int h, bool more) {
        const uint64_t v = v_desc + (step % kStages) * (kTileBytes<D> >> 4) + h * (D * 8);
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < kKeys / 32; i++)
                mma_ts(tm + 256 + half * D, tm + half * kKeys + h * (kKeys / 2) + i * 8, v + 2 * i, kIdO,
                       more || i > 0);
            mma_commit(bars + 8 * (kPvDone + 2 * half + h));
        }
        __syncwarp();
    };
    auto commit = [&](int bar) {
        if (elect_one())
            mma_commit(bars + 8 * bar);
        __syncwarp();
    };
    for (int s = 0; s < sh.n_segs; s++) {
        const Seg &sg = sh.segs[s];
        if (sg.tiles == 0)
            continue;
        const bool two = sg.tokens * p.group - sg.rt * kRows > 128;
        wait(sh, bars + 8 * kQFull, items & 1, p.v.status);
        items++;
        // Step j's scores beside step j - 1's outputs, by halves of the keys: while
        // the softmax of one half runs, the other half's products do.
        for (int j = 0; j <= sg.tiles; j++) {
            const uint32_t step = steps + j, before = step - 1;
            const bool scores = j < sg.tiles, outputs = j > 0;
            if (scores)
                wait(sh, bars + 8 * (kKFull + step % kStages), (step / kStages) & 1, p.v.status);
            if (outputs)
                wait(sh, bars + 8 * (kVFull + before % kStages), (before / kStages) & 1, p.v.status);
#pragma unroll
            for (int x = 0; x < 4; x++) {
                const int h = x >> 1, half = x & 1;
                if (half && !two)
                    continue;
                if (outputs) {
                    wait(sh, bars + 8 * (kPFull + 2 * half + h), cnt[half] & 1, p.v.status);
                    tc_fence_after();
                    output(half, before, h, j > 1 || h > 0);
                    cnt[half] += h;
                }
                if (scores) {
                    tc_fence_after();
                    score(half, step, h);
                }
            }
            if (outputs)
                commit(kVEmpty + before % kStages);
            if (scores)
                commit(kKEmpty + step % kStages);
            if (j == sg.tiles - 1)
                commit(kQEmpty);
        }
        steps += sg.tiles;
    }
    // every commit has arrived before the barriers go
    if (steps > 0)
        wait(sh, bars + 8 * (kVEmpty + (steps - 1) % kStages), ((steps - 1) / kStages) & 1, p.v.status);
}

template <int D>
__device__ __forceinline__ void unpack_role(const AttnParams &p, Shared &sh, uint32_t bars, uint32_t q_at,
                                            uint32_t k_at, uint32_t v_at, uint32_t &steps, uint32_t &items) {
    const Kv4View &v = p.v;
    const int t = threadIdx.x - kSoftmax, lane = t & 31;
    const Codes codes;
    const int64_t block = int64_t(D + 8) << v.page_log2, page_bytes = block * v.heads;
    const int mask = (1 << v.page_log2) - 1;
    // K: a key; V: a word (8 dimensions) of 8 keys, VT times
    constexpr int KC = D / 32;            // 16-byte chunks of a packed row
    constexpr int VW = D / 8;             // words of a packed row
    constexpr int VT = kKeys / 8 * VW / kUnpack, KG = kUnpack / VW;
    const int key = t, vw = t % VW, kg = t / VW;
    // Order of a V word's bytes and halves of a byte, so that eight lanes
    // write eight different rows (mod 8) at a time.
    uint32_t sel[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t b = (j + vw) & 3;
        sel[j] = b * 0x11u | (4 + b) * 0x1100u;
    }
    const bool odd_first = (vw >> 2) & 1;
    const uint32_t m_a = odd_first ? codes.mask4 : codes.mask0, m_b = odd_first ? codes.mask0 : codes.mask4;
    const uint32_t c_a = odd_first ? codes.mid4 : codes.mid0, c_b = odd_first ? codes.mid0 : codes.mid4;
    // Where the word's even (or odd) dimension of byte j goes in a V tile; the
    // other one is the next row (or the one before): 128 bytes and one chunk
    // bit on, both by exclusive or.  A second task lies a block of 64 keys on.
    static_assert(VT == 1 || KG == 8, "a thread's tasks lie in the same place of their blocks");
    uint32_t v_to[4];
    constexpr uint32_t v_flip = 128u ^ 16u;
#pragma unroll
    for (int j = 0; j < 4; j++)
        v_to[j] = tile_at(8 * vw + 2 * ((j + vw) & 3) + odd_first, kg, D);
    const float a_up = p.c1 * kQDown;
    for (int s = 0; s < sh.n_segs; s++) {
        const Seg &sg = sh.segs[s];
        if (sg.tiles == 0)
            continue;
        const int r0 = sg.rt * kRows, rows = sg.tokens * p.group;
        const uint8_t *const base = v.pages + sg.head * block;
        const int32_t *const table = v.table + int64_t(sg.s) * v.table_stride;
        uint4 rk[KC];
        uint32_t rv[VT][8], rp[2];
        int pk, pv[VT];
        auto page_of = [&](int at) { return __ldg(table + (min(max(at, sg.lo), sg.len - 1) >> v.page_log2)); };
        auto pages = [&](int key0) {
            pk = page_of(key0 + key);
#pragma unroll
            for (int n = 0; n < VT; n++)
                pv[n] = page_of(key0 + 8 * (kg + n * KG));
        };
        auto bad = [&](int page) {
            if (uint32_t(page) < uint32_t(v.n_pages))
                return false;
            atomicOr(v.status, kStatusBadCache);
            return true;
        };
        // A key or eight keys of V that are not there are zeros; pages are
        // looked at here, a tile after they were loaded.
        auto load_k = [&](int key0) {
            const int at = key0 + key;
#pragma unroll
            for (int i = 0; i < KC; i++)
                rk[i] = make_uint4(0, 0, 0, 0);
            rp[0] = rp[1] = 0;
            if (!bad(pk) && at < sg.len) {
                const uint8_t *b = base + pk * page_bytes;
                const uint4 *src = reinterpret_cast<const uint4 *>(b + (at & mask) * (D / 2));
#pragma unroll
                for (int i = 0; i < KC; i++)
                    rk[i] = __ldg(src + i);
                const uint8_t *par = b + kv4_params<D>(v.page_log2, at & mask, 0);
                rp[0] = __ldg(reinterpret_cast<const uint32_t *>(par));
                rp[1] = __ldg(reinterpret_cast<const uint32_t *>(par + (4 << v.page_log2)));
            }
        };
        auto load_v = [&](int key0) {
#pragma unroll
            for (int n = 0; n < VT; n++) {
                const int at = key0 + 8 * (kg + n * KG);
                const uint8_t *b = base + pv[n] * page_bytes + kv4_codes<D>(v.page_log2, at & mask, 1) + vw * 4;
                if (!bad(pv[n]) && sg.len - at >= 8) {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        rv[n][i] = __ldg(reinterpret_cast<const uint32_t *>(b + i * (D / 2)));
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        rv[n][i] = uint32_t(pv[n]) < uint32_t(v.n_pages) && at + i < sg.len
                                       ? __ldg(reinterpret_cast<const uint32_t *>(b + i * (D / 2)))
                                       : 0u;
                }
            }
        };
        const int first = sg.first * kKeys;
        pages(first);

        // queries: a thread writes two rows, in the order the codes of a word come out in
        wait(sh, bars + 8 * kQEmpty, (items & 1) ^ 1, v.status);
        for (int rr = t; rr < kRows; rr += kUnpack) {
            const bool in = rr < rows - r0;
            const int i = p.by_group.of(in ? r0 + rr : 0);
            const int64_t tok = sg.t0 + i, head = sg.head * p.group + (r0 + rr - i * p.group);
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q.p + tok * p.q.ts + head * p.q.hs);
            const uint32_t to = q_at + (rr >> 7) * kTileBytes<D>;
            float sum = 0.f;
#pragma unroll 8
            for (int c = 0; c < D / 8; c++) {
                const uint4 x = in ? src[c] : make_uint4(0, 0, 0, 0);
                const uint32_t a[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; k++)
                    sum += bf16_lo(a[k]) + bf16_hi(a[k]);
                sts128(to + tile_at(rr & 127, c, 128), mul2_bf16(__byte_perm(x.x, x.z, 0x5410), kQUpLow),
                       mul2_bf16(__byte_perm(x.x, x.z, 0x7632), kQUpHigh),
                       mul2_bf16(__byte_perm(x.y, x.w, 0x5410), kQUpLow),
                       mul2_bf16(__byte_perm(x.y, x.w, 0x7632), kQUpHigh));
            }
            sh.qs[items & 1][rr] = sum;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bars + 8 * kQFull);
        items++;
        load_k(first);
        load_v(first);
        if (sg.tiles > 1)
            pages(first + kKeys);

        for (int j = 0; j < sg.tiles; j++, steps++) {
            const uint32_t stage = steps % kStages, turn = (steps / kStages) & 1, par = steps % kParStages;
            const bool more = j + 1 < sg.tiles;
            {
                float *const kd = reinterpret_cast<float *>(sh.kpar[par]) + (key >> 1) * 4 + (key & 1);
                float *const vd = reinterpret_cast<float *>(sh.vpar[par]) + (key >> 1) * 4 + (key & 1);
                kd[0] = bf16_lo(rp[0]) * a_up;
                kd[2] = bf16_hi(rp[0]) * p.c1;
                vd[0] = bf16_lo(rp[1]) * kPUp;
                vd[2] = fmaf(8.f, bf16_lo(rp[1]), bf16_hi(rp[1]));
            }
            wait(sh, bars + 8 * (kKEmpty + stage), turn ^ 1, v.status);
            const uint32_t kt = k_at + stage * kTileBytes<D>;
#pragma unroll
            for (int i = 0; i < KC; i++) {
                const uint32_t a[4] = {rk[i].x, rk[i].y, rk[i].z, rk[i].w};
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint32_t y = a[k] >> 8;
                    sts128(kt + tile_at(key, i * 4 + k, kKeys), codes.low(a[k]), codes.high(a[k]),
                           codes.low(y), codes.high(y));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bars + 8 * (kKFull + stage));
                mbar_arrive(bars + 8 * (kParFull + par));
            }
            if (more)
                load_k(first + (j + 1) * kKeys);
            wait(sh, bars + 8 * (kVEmpty + stage), turn ^ 1, v.status);
            const uint32_t vt = v_at + stage * kTileBytes<D>;
#pragma unroll
            for (int n = 0; n < VT; n++)
#pragma unroll
                for (int jj = 0; jj < 4; jj++) {
                    uint32_t e[4];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        e[i] = __byte_perm(rv[n][2 * i], rv[n][2 * i + 1], sel[jj]);
                    const uint32_t to = vt + v_to[jj] + n * (D * 128);
                    sts128(to, sub2(e[0] & m_a, c_a), sub2(e[1] & m_a, c_a), sub2(e[2] & m_a, c_a),
                           sub2(e[3] & m_a, c_a));
                    sts128(to ^ v_flip, sub2(e[0] & m_b, c_b), sub2(e[1] & m_b, c_b), sub2(e[2] & m_b, c_b),
                           sub2(e[3] & m_b, c_b));
                }
            if (more) {
                load_v(first + (j + 1) * kKeys);
                if (j + 2 < sg.tiles)
                    pages(first + (j + 2) * kKeys);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bars + 8 * (kVFull + stage));
        }
    }
}

template <int D>
__device__ __forceinline__ void softmax_role(const AttnParams &p, Shared &sh, uint32_t bars, uint64_t total,
                                             uint32_t workers, uint64_t cut0, uint32_t &steps, uint32_t &items,
                                             uint32_t &cnt) {
    constexpr int PF = kRows * (D + 2);
    const int half = threadIdx.x >> 7, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t s_tm = sh.tmem + lanes + half * kKeys, o_tm = sh.tmem + lanes + 256 + half * D;
    // The lower half passes over items of up to 128 rows without a wait and may then be
    // steps ahead of the unpack warps, where the parity of kParFull tells nothing: it
    // waits for its next item's first scores before that (done for every item, a chunk
    // of 1024 tokens after 15360 with two short ones takes 352 us instead of 344).
    bool ahead = false;
    for (int sgi = 0; sgi < sh.n_segs; sgi++) {
        const Seg &sg = sh.segs[sgi];
        const int r0 = sg.rt * kRows, rows = sg.tokens * p.group;
        const int r = r0 + int(threadIdx.x);
        const bool active = r0 + 128 * half < rows;  // this half has rows
        const Seq sq{sg.t0, sg.tokens, sg.len};
        // The warp's 32 rows lie like the rows of a matrix product's fragment: a
        // thread has rows g + 8 i (i < 4) and of them the key pairs 8 k + 2 t, so that a
        // pair's scales and offsets are read once for four rows.
        float m[4], lim[4];      // maximum; the sum of 16 probabilities from which it is raised
        uint64_t mm[4], qs[4];   // less the maximum, and the sum of q, in pairs
        uint64_t l2[4], z2[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            m[i] = -INFINITY;
            lim[i] = -1.f;       // no maximum yet: any sum
            l2[i] = z2[i] = mm[i] = qs[i] = 0;
        }
        if (ahead && active && sg.tiles > 0) {
            wait(sh, bars + 8 * (kSFull + 2 * half), cnt & 1, p.v.status);
            ahead = false;
        }
        for (int j = 0; j < sg.tiles; j++) {
            const uint32_t step = steps + j, par = step % kParStages;
            if (!active)
                continue;
            const int key0 = (sg.first + j) * kKeys;
            wait(sh, bars + 8 * (kParFull + par), (step / kParStages) & 1, p.v.status);
            if (j == 0) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float q = sh.qs[items & 1][32 * warp + g + 8 * i];
                    qs[i] = pair2(q, q);
                }
            }
            const bool open = key0 < sg.all_lo || sg.all_hi - key0 < kKeys;  // (key0 + kKeys may be 2^31)
            auto tile = [&](auto masked) {
                constexpr bool kOpen = decltype(masked)::value;
                int lo[4], hi[4];  // the rows' keys in this tile, less the thread's first
                if constexpr (kOpen) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int tok = p.by_group.of(min(r0 + 32 * warp + g + 8 * i, rows - 1));
                        const KeyRange kr = visible(p, sq, tok, tok);
                        lo[i] = kr.lo - key0 - 2 * t;
                        hi[i] = min(kr.hi, sg.len) - key0 - 2 * t;
                    }
                }
                const ulonglong2 *const kp = reinterpret_cast<const ulonglong2 *>(sh.kpar[par]) + t;
                const ulonglong2 *const vp = reinterpret_cast<const ulonglong2 *>(sh.vpar[par]) + t;
#pragma unroll 1
                for (int h = 0; h < 2; h++) {  // halves of the keys; P of one lies over its scores
                    wait(sh, bars + 8 * (kSFull + 2 * half + h), cnt & 1, p.v.status);
                    tc_fence_after();
                    uint64_t y[4][8], sum[4];  // [row][key group]: scores, then probabilities
                    for (bool again = false;; again = true) {
                        uint32_t x[64];  // [32 keys][16 rows' half][key group][row g, g + 8][pair]
#pragma unroll
                        for (int c = 0; c < 4; c++)
                            tmem_ld_16x256_x4(s_tm + 64 * h + 32 * (c >> 1) + (uint32_t(16 * (c & 1)) << 16),
                                              x + 16 * c);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 8; k++) {
                            const ulonglong2 ab = kp[32 * h + 4 * k];
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const uint32_t *const w = x + 32 * (k >> 2) + 16 * (i >> 1) + 4 * (k & 3) + 2 * (i & 1);
                                y[i][k] = fma2(pair2(__uint_as_float(w[0]), __uint_as_float(w[1])), ab.x,
                                               fma2(ab.y, qs[i], mm[i]));
                                if constexpr (kOpen) {
                                    const float2 f = unpair(y[i][k]);
                                    const int at = 64 * h + 8 * k;
                                    y[i][k] = pair2(at >= lo[i] && at < hi[i] ? f.x : -INFINITY,
                                                    at + 1 >= lo[i] && at + 1 < hi[i] ? f.y : -INFINITY);
                                }
                            }
                        }
                        if (again) {
                            // Raise the maxima to those of these keys: what the rows have so far
                            // is scaled down.
                            float f[4];
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                float top = -INFINITY;
#pragma unroll
                                for (int k = 0; k < 8; k++) {
                                    const float2 v = unpair(y[i][k]);
                                    top = fmaxf(top, fmaxf(v.x, v.y));
                                }
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                                const float m0 = m[i] == -INFINITY ? 0.f : m[i];
                                const float m2 = fmaxf(m[i], m0 + top), m20 = m2 == -INFINITY ? 0.f : m2;
                                f[i] = m[i] == -INFINITY ? 0.f : exp2_fast(m[i] - m20);
                                const uint64_t ff = pair2(f[i], f[i]), d = pair2(m0 - m20, m0 - m20);
                                l2[i] = mul2(l2[i], ff);
                                z2[i] = mul2(z2[i], ff);
#pragma unroll
                                for (int k = 0; k < 8; k++)
                                    y[i][k] = add2(y[i][k], d);
                                m[i] = m2;
                                mm[i] = pair2(-m20, -m20);
                                lim[i] = m2 == -INFINITY ? -1.f : kRaise;
                            }
                            if (j > 0 || h > 0) {
                                // the output has a row a thread
                                float fo = 0.f;
#pragma unroll
                                for (int i = 0; i < 4; i++) {
                                    const float o = __shfl_sync(0xffffffffu, f[i], 4 * (lane & 7));
                                    fo = (lane >> 3) == i ? o : fo;
                                }
                                wait(sh, bars + 8 * (kPvDone + 2 * half + (h ^ 1)), (cnt + h - 1) & 1, p.v.status);
                                tc_fence_after();
#pragma unroll 1
                                for (int d0 = 0; d0 < D; d0 += 16) {
                                    uint32_t w[16];
                                    tmem_ld16(o_tm + d0, w);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int i = 0; i < 16; i++)
                                        w[i] = __float_as_uint(__uint_as_float(w[i]) * fo);
                                    tmem_st16(o_tm + d0, w);
                                }
                            }
                        }
                        uint64_t pr[4][8];
                        bool raise = false;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
#pragma unroll
                            for (int k = 0; k < 8; k++) {
                                const float2 f = unpair(y[i][k]);
                                pr[i][k] = pair2(exp2_fast(f.x), exp2_fast(f.y));
                            }
                            sum[i] = add2(add2(add2(pr[i][0], pr[i][1]), add2(pr[i][2], pr[i][3])),
                                          add2(add2(pr[i][4], pr[i][5]), add2(pr[i][6], pr[i][7])));
                            const float2 f = unpair(sum[i]);
                            raise = raise || f.x + f.y > lim[i];
                        }
#pragma unroll
                        for (int i = 0; i < 4; i++)
#pragma unroll
                            for (int k = 0; k < 8; k++)
                                y[i][k] = pr[i][k];
                        if (again || !__any_sync(0xffffffffu, raise))
                            break;
                    }
                    uint32_t pk[32];  // [32 keys][16 rows' half][key group][row g, g + 8]
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        l2[i] = add2(l2[i], sum[i]);
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const ulonglong2 sm = vp[32 * h + 4 * k];
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            uint64_t ps = mul2(y[i][k], sm.x);
                            if constexpr (kOpen) {  // a masked key's scale may be anything
                                const int at = 64 * h + 8 * k;
                                const float2 a = unpair(ps), b = unpair(mul2(y[i][k], sm.y));
                                const bool in0 = at >= lo[i] && at < hi[i], in1 = at + 1 >= lo[i] && at + 1 < hi[i];
                                ps = pair2(in0 ? a.x : 0.f, in1 ? a.y : 0.f);
                                z2[i] = add2(z2[i], pair2(in0 ? b.x : 0.f, in1 ? b.y : 0.f));
                            } else {
                                z2[i] = fma2(y[i][k], sm.y, z2[i]);
                            }
                            const float2 a = unpair(ps);
                            pk[16 * (k >> 2) + 8 * (i >> 1) + 2 * (k & 3) + (i & 1)] = bf16_pack(a.x, a.y);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        tmem_st_16x128_x4(s_tm + 64 * h + 16 * (c >> 1) + (uint32_t(16 * (c & 1)) << 16), pk + 8 * c);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bars + 8 * (kPFull + 2 * half + h));
                }
            };
            if (open)
                tile(std::true_type());
            else
                tile(std::false_type());
            cnt++;
        }
        ahead = ahead || !active;
        steps += sg.tiles;
        items += sg.tiles > 0;

        // From here on a thread has one row: its maximum and sums from the four
        // threads that had them.
        float row_m = 0.f, l = 0.f, z = 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 lf = unpair(l2[i]), zf = unpair(z2[i]);
            float ls = lf.x + lf.y, zs = zf.x + zf.y;
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                ls += __shfl_xor_sync(0xffffffffu, ls, o);
                zs += __shfl_xor_sync(0xffffffffu, zs, o);
            }
            const float mi = __shfl_sync(0xffffffffu, m[i], 4 * (lane & 7));
            ls = __shfl_sync(0xffffffffu, ls, 4 * (lane & 7));
            zs = __shfl_sync(0xffffffffu, zs, 4 * (lane & 7));
            if ((lane >> 3) == i) {
                row_m = mi;
                l = ls;
                z = zs;
            }
        }
        const bool whole = sg.tiles == sg.of, valued = active && sg.tiles > 0;
        const int slot = cut0 > sg.u0 ? 0 : 1;
        float *const part = p.parts + (2 * uint64_t(blockIdx.x) + slot) * PF;
        if (valued) {
            wait(sh, bars + 8 * (kPvDone + 2 * half + 1), (cnt - 1) & 1, p.v.status);
            tc_fence_after();
        }
        if (active) {
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {
                uint32_t w[2][16];
#pragma unroll
                for (int i = 0; i < 16; i++)
                    w[0][i] = w[1][i] = 0;
                if (valued) {
                    tmem_ld16(o_tm + d0, w[0]);
                    tmem_ld16(o_tm + d0 + 16, w[1]);
                    tmem_ld_wait();
                }
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; i++)
                    o[i] = fmaf(__uint_as_float(w[i / 16][i % 16]), i & 1 ? kPDownHigh : kPDownLow, z);
                if (r < rows) {
                    if (whole) {
                        store_dims<32>(p, sg.t0, sg.head, r, d0, o, row_m, l);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            reinterpret_cast<float4 *>(part)[(d0 / 4 + i) * kRows + threadIdx.x] =
                                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
            }
            if (!whole) {
                part[kRows * D + threadIdx.x] = row_m;
                part[kRows * D + kRows + threadIdx.x] = l;
            }
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
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(const AttnParams p) {
    using S = Sched<kRows, kKeys, kItemCost>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t raw = smem_addr(smem_raw), q_at = (raw + 1023u) & ~1023u;
    const uint32_t k_at = q_at + 2 * kTileBytes<D>, v_at = k_at + kStages * kTileBytes<D>;
    const uint32_t bars = smem_addr(sh.bars);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; i++) {
            uint32_t n = 1;  // a commit
            if (i == kQFull || (i >= kKFull && i < kKEmpty) || (i >= kVFull && i < kVEmpty) ||
                (i >= kParFull && i < kSFull))
                n = kUnpack / 32;
            else if (i >= kPFull && i < kPvDone)
                n = 4;
            mbar_init(bars + 8 * i, n);
        }
        mbar_init_fence();
        sh.dead = 0;
    }
    grid_dep_launch();
    grid_dep_wait();
    const uint64_t total = build_row<S, kThreads, true>(p, sh.row);
    const uint32_t workers = uint32_t(min((total + kMinShare - 1) / kMinShare, uint64_t(gridDim.x)));
    if (blockIdx.x >= workers)
        return;
    if (warp == kThreads / 32 - 1)
        tmem_alloc(smem_addr(&sh.tmem), kTmemCols);
    const uint64_t cut0 = mul_div(total, blockIdx.x, workers), cut1 = mul_div(total, blockIdx.x + 1, workers);
    // From here on every role walks through the lists of segments by itself;
    // barrier 0 stands before and after a list's work.  Registers a thread by
    // warpgroup: 2 x 176 + 104 + 56 = 4 x 128, the launch's.
    tc_fence_before();
    if (warp < kSoftmax / 32) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        Item it{};
        if (warp == 0)
            it = locate<S>(p, sh.row, cut0);
        uint32_t steps = 0, items = 0, cnt = 0;
        for (uint64_t u = cut0; u < cut1;) {
            if (warp == 0) {
                int n;
                const uint64_t to = list_segments<S, kSegs>(p, it, u, cut1, sh.segs, &n);
                if (lane == 0) {
                    sh.listed_to = to;
                    sh.n_segs = n;
                }
            }
            __syncthreads();
            tc_fence_after();
            u = sh.listed_to;
            softmax_role<D>(p, sh, bars, total, workers, cut0, steps, items, cnt);
            __syncthreads();
        }
    } else if (warp < (kSoftmax + kUnpack) / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        uint32_t steps = 0, items = 0;
        for (uint64_t u = cut0; u < cut1;) {
            __syncthreads();
            u = sh.listed_to;
            unpack_role<D>(p, sh, bars, q_at, k_at, v_at, steps, items);
            __syncthreads();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        uint32_t steps = 0, items = 0, cnt[2] = {0, 0};
        for (uint64_t u = cut0; u < cut1;) {
            __syncthreads();
            tc_fence_after();
            u = sh.listed_to;
            if (warp == (kSoftmax + kUnpack) / 32)
                mma_role<D>(p, sh, bars, q_at, k_at, v_at, steps, cnt, items);
            __syncthreads();
        }
    }
    if (warp == kThreads / 32 - 1)
        tmem_dealloc(sh.tmem, kTmemCols);
}

template <int D>
uw_status launch(const AttnParams &p, int ctas, cudaStream_t st) {
    if (!ensure_smem(kv4_prefill_kernel<D>, kSmem<D>))
        return UW_ERR_CUDA;
    return launch_overlapped(kv4_prefill_kernel<D>, dim3(unsigned(ctas)), dim3(kThreads), kSmem<D>, st, p) ==
                   cudaSuccess
               ? UW_OK
               : UW_ERR_CUDA;
}

}  // namespace

int kv4_prefill_ctas() { return sm_count(); }

size_t kv4_prefill_part_floats(int head_dim) { return 2 * size_t(kv4_prefill_ctas()) * kRows * (head_dim + 2); }

uw_status launch_kv4_prefill(const AttnParams &p, int head_dim, cudaStream_t st) {
    const int n = kv4_prefill_ctas();
    return head_dim == 128 ? launch<128>(p, n, st) : launch<64>(p, n, st);
}

}  // namespace uw
