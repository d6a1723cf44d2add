// What the attention kernels over the 4-bit paged cache share: their
// parameters, the cut of the work into equal shares, and the joining of the
// shares of one item.
//
// An item is one (sequence, kv head, row tile): the rows of the tile are the
// new tokens' query heads that read this kv head, row r = token r / group,
// head r % group.  Its units are the key tiles that its rows can see, in
// order, and a few more for what an item costs however short it is.  All items'
// units in a row (sequence by sequence, head by head, tile by tile) are cut
// into shares of equal length, so that any mix of lengths fills the GPU.  Every
// CTA finds its share from the lengths on the device: nothing is planned on
// the host and a captured launch replays with other lengths.
//
// An item that lies in several shares is joined by the CTA that finishes last:
// each part leaves its unnormalised output, maximum and sum in the workspace,
// and the parts are added in their order, so the same call gives the same
// bits whichever CTA joins.  A share has at most two parts of such items (the
// end of one that began before, the beginning of one that goes on).
#pragma once
#include "kv4.cuh"

namespace uw {

// Division by a number that the host knows: n / d for 0 <= n < 2^31 as
// n * ceil(2^(31 + s) / d) >> (31 + s) with 2^s >= d.
struct Divisor {
    uint32_t d, mul, shift;
    Divisor(uint32_t d = 1) : d(d), shift(31) {
        while ((1ull << (shift - 31)) < d)
            shift++;
        mul = uint32_t(((1ull << shift) + d - 1) / d);
    }
    __device__ __forceinline__ int of(int n) const { return int((uint64_t(uint32_t(n)) * mul) >> shift); }
};

struct AttnParams {
    Kv4View v;
    Rows q, o;
    float *lse;
    float c1;                 // softmax scale * log2(e)
    int32_t q_heads, group, causal, window;
    Divisor by_group;
    bool out32;               // rows of o begin on 32-byte steps
    int32_t rows_min, rows_max;  // sequences with rows (new * group) in this range are this launch's
    float *parts;             // parts of RB * (D + 2) floats: output, maximum, sum
    uint32_t *counters;       // [gridDim.x], left at zero
};

// Keys [lo, hi) that some row of tokens [i0, i1] of a sequence sees.  (Of more
// new tokens than the sequence holds the first have negative positions, and
// a window may be any number: nothing is subtracted from a negative one.)
struct KeyRange {
    int32_t lo, hi;
};
__device__ __forceinline__ KeyRange visible(const AttnParams &p, const Seq &s, int i0, int i1) {
    const int32_t before = s.len - s.n;
    const int32_t hi = p.causal ? before + i1 + 1 : s.len;
    const int32_t lo = p.window ? max(before + i0 + 1, 0) - p.window : 0;
    return {max(lo, 0), max(hi, 0)};
}

// One item's place in the row of units.
struct Item {
    int s, head, rt;
    Seq q;
    KeyRange keys;
    uint64_t u0;     // its first unit
    uint32_t tiles;  // its key tiles: the first of its units
    uint32_t n;      // its units
};

template <int RB, int T, int kCost>  // rows of a row tile, keys of a unit, units an item costs beyond its tiles
struct Sched {
    static constexpr int kRows = RB, kKeys = T;
    static __device__ __forceinline__ bool mine(const AttnParams &p, const Seq &s) {
        const int32_t rows = s.n * p.group;
        return rows >= p.rows_min && rows <= p.rows_max && rows > 0;
    }
    static __device__ __forceinline__ int row_tiles(const AttnParams &p, const Seq &s) {
        return (s.n * p.group - 1) / RB + 1;
    }
    static __device__ __forceinline__ KeyRange tile_keys(const AttnParams &p, const Seq &s, int rt) {
        const int32_t r0 = rt * RB, r1 = r0 + min(RB, s.n * p.group - r0) - 1;
        return visible(p, s, p.by_group.of(r0), p.by_group.of(r1));
    }
    static __device__ __forceinline__ uint32_t tiles(const KeyRange &k) {
        return k.hi > k.lo ? uint32_t((k.hi - 1) / T - k.lo / T + 1) : 0u;
    }
    // Units of one head of a sequence: by one thread, and by a warp that
    // shares its row tiles.
    static __device__ __forceinline__ uint64_t seq_units(const AttnParams &p, const Seq &s) {
        if (!mine(p, s))
            return 0;
        uint64_t n = 0;
        const int rts = row_tiles(p, s);
        for (int rt = 0; rt < rts; rt++)
            n += kCost + tiles(tile_keys(p, s, rt));
        return n;
    }
    static __device__ __forceinline__ uint64_t seq_units_warp(const AttnParams &p, const Seq &s) {
        if (!mine(p, s))
            return 0;
        const int rts = row_tiles(p, s);
        if (rts == 1)
            return kCost + tiles(tile_keys(p, s, 0));
        uint64_t n = 0;
        for (int rt = threadIdx.x & 31; rt < rts; rt += 32)
            n += kCost + tiles(tile_keys(p, s, rt));
#pragma unroll
        for (int o = 16; o; o >>= 1)
            n += __shfl_xor_sync(0xffffffffu, n, o);
        return n;
    }
    static __device__ __forceinline__ void set_tile(const AttnParams &p, Item &it, int rt) {
        it.rt = rt;
        it.keys = tile_keys(p, it.q, rt);
        it.tiles = tiles(it.keys);
        it.n = kCost + it.tiles;
    }
};

// The row of units as a CTA of kThreads threads sees it: thread i stands for
// the sequences [i * per, (i + 1) * per), before[i] units come before them.
template <int kThreads>
struct Row {
    uint64_t before[kThreads], sums[kThreads / 32];
    Seq seq[kThreads];  // with per = 1: the sequence
};

// Fills the row (all threads call); returns all units.  kWide: a warp for
// each sequence, its lanes for the row tiles, where sequences have many;
// otherwise a thread for each sequence.
template <class S, int kThreads, bool kWide>
__device__ __forceinline__ uint64_t build_row(const AttnParams &p, Row<kThreads> &row) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.v.n_seqs + kThreads - 1) / kThreads;
    uint64_t mine = 0;
    if constexpr (kWide) {
        row.before[threadIdx.x] = 0;
        __syncthreads();
        for (int s0 = 0; s0 < p.v.n_seqs; s0 += kThreads) {
            const int own = s0 + warp + lane * kWarps;  // the lane's sequence, of this warp's 32
            const Seq q = own < p.v.n_seqs ? kv4_seq(p.v, own) : Seq{0, 0, 0};
            if (own < p.v.n_seqs)
                row.seq[own % kThreads] = q;
            for (int k = 0; k < 32 && s0 + warp + k * kWarps < p.v.n_seqs; k++) {
                const Seq one{__shfl_sync(0xffffffffu, q.t0, k), __shfl_sync(0xffffffffu, q.n, k),
                              __shfl_sync(0xffffffffu, q.len, k)};
                const uint64_t u = S::seq_units_warp(p, one) * p.v.heads;
                if (lane == 0 && u)
                    atomicAdd(reinterpret_cast<unsigned long long *>(&row.before[(s0 + warp + k * kWarps) / per]), u);
            }
        }
        __syncthreads();
        mine = row.before[threadIdx.x];
    } else {
        const int a = min(int(threadIdx.x) * per, p.v.n_seqs), b = min(a + per, p.v.n_seqs);
        for (int s = a; s < b; s++) {
            const Seq q = kv4_seq(p.v, s);
            mine += S::seq_units(p, q) * p.v.heads;
            row.seq[threadIdx.x] = q;
        }
    }
    uint64_t v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += u;
    }
    if (lane == 31)
        row.sums[warp] = v;
    __syncthreads();
    uint64_t before = v - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        const uint64_t t = row.sums[w];
        before += w < warp ? t : 0;
        all += t;
    }
    row.before[threadIdx.x] = before;
    __syncthreads();
    return all;
}

// a * b / c and a / b, in 32 bits where they fit (a 64-bit division is a
// hundred instructions one after the other).
__device__ __forceinline__ uint64_t mul_div(uint64_t a, uint32_t b, uint32_t c) {
    const uint64_t ab = a * b;
    return (ab >> 32) == 0 ? uint32_t(ab) / c : ab / c;
}
__device__ __forceinline__ uint64_t divide(uint64_t a, uint64_t b) {
    return ((a | b) >> 32) == 0 ? uint32_t(a) / uint32_t(b) : a / b;
}

// The item that holds unit u (of fewer than all); a warp calls.
template <class S, int kThreads>
__device__ __forceinline__ Item locate(const AttnParams &p, const Row<kThreads> &row, uint64_t u) {
    const int lane = threadIdx.x & 31;
    const int per = (p.v.n_seqs + kThreads - 1) / kThreads;
    int i = -1;  // the last thread with before <= u
#pragma unroll 1
    for (int k = 0; k < kThreads / 32 && 32 * k * per < p.v.n_seqs; k++)
        i += __popc(__ballot_sync(0xffffffffu, row.before[32 * k + lane] <= u));
    Item it;
    it.s = i * per;
    uint64_t rest = u - row.before[i], per_head;
    it.u0 = row.before[i];
    if (per == 1) {
        it.q = row.seq[i];
        per_head = S::seq_units_warp(p, it.q);
    } else {
        for (;; it.s++) {
            it.q = kv4_seq(p.v, it.s);
            per_head = S::seq_units_warp(p, it.q);
            if (rest < per_head * p.v.heads)
                break;
            rest -= per_head * p.v.heads;
            it.u0 += per_head * p.v.heads;
        }
    }
    it.head = int(divide(rest, per_head));
    rest -= it.head * per_head;
    it.u0 += it.head * per_head;
    const int rts = S::row_tiles(p, it.q);
    if (rts == 1) {
        S::set_tile(p, it, 0);
        return it;
    }
    // its row tile: 32 of them at a time
    for (int rt0 = 0;; rt0 += 32) {
        const int rt = rt0 + lane;
        uint32_t n = 0;
        if (rt < rts) {
            S::set_tile(p, it, rt);
            n = it.n;
        }
        uint64_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o)
                upto += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, rt < rts && rest < upto);
        if (past) {
            const int at = __ffs(past) - 1;
            it.u0 += __shfl_sync(0xffffffffu, upto - n, at);
            S::set_tile(p, it, rt0 + at);
            return it;
        }
        const uint64_t all = __shfl_sync(0xffffffffu, upto, 31);
        rest -= all;
        it.u0 += all;
    }
}

// A share's part of one item: tiles first .. first + tiles - 1.
struct Seg {
    uint64_t u0;
    int32_t s, head, rt, t0, tokens, len;
    int32_t first, tiles, of;  // `of`: the item's tiles
    int32_t lo;                // the first key that some row sees: pages before its page are not looked at
    int32_t all_lo, all_hi;    // keys that every row sees
};
// A warp lists the segments of the units from u (in item `it`) up to `end`,
// at most kMost of them; returns the unit after them and leaves `it` there.
// An item's last units, which are no tiles, are nobody's; one that sees no
// key at all is a segment without tiles of the share that has its first unit.
// The sequences' lengths are read 32 at a time.  `segs` may be a list that
// the warp has just worked through.
template <class S, int kMost>
__device__ __forceinline__ uint64_t list_segments(const AttnParams &p, Item &it, uint64_t u, uint64_t end, Seg *segs,
                                                  int *count) {
    const int lane = threadIdx.x & 31;
    int base = it.s, n = 0;
    Seq next{0, 0, 0};
    bool loaded = false;
    __syncwarp();  // every lane has read the list before
    while (u < end && n < kMost) {
        const uint32_t a = uint32_t(u - it.u0), b = uint32_t(min(end - it.u0, uint64_t(it.n)));
        const int tiles = int(min(b, it.tiles)) - int(a);
        if (tiles > 0 || (it.tiles == 0 && a == 0)) {
            if (lane == 0) {
                Seg g;
                g.u0 = it.u0;
                g.s = it.s;
                g.head = it.head;
                g.rt = it.rt;
                g.t0 = it.q.t0;
                g.tokens = it.q.n;
                g.len = it.q.len;
                g.first = it.keys.lo / S::kKeys + int(a);
                g.tiles = max(tiles, 0);
                g.of = int(it.tiles);
                g.lo = it.keys.lo;
                const int r0 = it.rt * S::kRows, r1 = r0 + min(S::kRows, it.q.n * p.group - r0) - 1;
                const int i0 = p.by_group.of(r0), i1 = p.by_group.of(r1);
                g.all_lo = visible(p, it.q, i1, i1).lo;
                g.all_hi = min(visible(p, it.q, i0, i0).hi, it.q.len);
                segs[n] = g;
            }
            n++;
        }
        u = it.u0 + b;
        if (u < end) {  // the next item
            it.u0 = u;
            int rt = it.rt + 1;
            if (rt == S::row_tiles(p, it.q)) {
                rt = 0;
                if (++it.head == p.v.heads) {
                    it.head = 0;
                    do {
                        if (!loaded || ++it.s - base == 32) {
                            it.s += loaded ? 0 : 1;
                            loaded = true;
                            base = it.s;
                            next = base + lane < p.v.n_seqs ? kv4_seq(p.v, base + lane) : Seq{0, 0, 0};
                        }
                        it.q.t0 = __shfl_sync(0xffffffffu, next.t0, it.s - base);
                        it.q.n = __shfl_sync(0xffffffffu, next.n, it.s - base);
                        it.q.len = __shfl_sync(0xffffffffu, next.len, it.s - base);
                    } while (!S::mine(p, it.q));
                }
            }
            S::set_tile(p, it, rt);
        }
    }
    *count = n;
    __syncwarp();
    return u;
}

// The share (of `workers` equal ones) that holds unit u: the last c with
// total * c / workers <= u.
__device__ __forceinline__ uint32_t share_of(uint64_t u, uint64_t total, uint32_t workers) {
    return uint32_t(divide((u + 1) * workers - 1, total));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A further part of a row (sum l2, unnormalised output o2) added to (l, o),
// scaled down by f to the joint maximum.
__device__ __forceinline__ void join_scaled(float &l, float4 &o, float f, float l2, float4 o2) {
    l = fmaf(f, l2, l);
    o.x = fmaf(f, o2.x, o.x);
    o.y = fmaf(f, o2.y, o.y);
    o.z = fmaf(f, o2.z, o.z);
    o.w = fmaf(f, o2.w, o.w);
}

// Four dimensions (4c ..) of row r of the items of a sequence (first token t0)
// and kv head: out = o / l, and with c = 0 the lse.
template <int D>
__device__ __forceinline__ void store_row(const AttnParams &p, int t0, int kv_head, int r, int c, float4 o, float m,
                                          float l) {
    const int i = p.by_group.of(r);
    const int64_t tok = t0 + i, head = kv_head * p.group + (r - i * p.group);
    const float inv = l == 0.f ? 0.f : 1.f / l;  // no key: o is 0 and stays 0
    *reinterpret_cast<uint2 *>(p.o.p + tok * p.o.ts + head * p.o.hs + 4 * c) =
        make_uint2(bf16_pack(o.x * inv, o.y * inv), bf16_pack(o.z * inv, o.w * inv));
    if (p.lse && c == 0)
        p.lse[tok * p.q_heads + head] = l == 0.f ? -INFINITY : 0.69314718056f * (m + log2f(l));
}

// The same for N dimensions from d0 on, a row a thread: where rows begin on 32-byte
// steps a store takes a whole sector (a prompt of 8192 tokens 653 us, by 16 bytes 666).
template <int N>
__device__ __forceinline__ void store_dims(const AttnParams &p, int t0, int kv_head, int r, int d0, const float (&o)[N],
                                           float m, float l) {
    const int i = p.by_group.of(r);
    const int64_t tok = t0 + i, head = kv_head * p.group + (r - i * p.group);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *const dst = p.o.p + tok * p.o.ts + head * p.o.hs + d0;
#pragma unroll
    for (int k = 0; k < N / 16; k++) {
        uint32_t a[8];
#pragma unroll
        for (int x = 0; x < 8; x++)
            a[x] = bf16_pack(o[16 * k + 2 * x] * inv, o[16 * k + 2 * x + 1] * inv);
        if (p.out32) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                         :: "l"(dst + 16 * k), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(a[4]), "r"(a[5]),
                            "r"(a[6]), "r"(a[7])
                         : "memory");
        } else {
            *reinterpret_cast<uint4 *>(dst + 16 * k) = make_uint4(a[0], a[1], a[2], a[3]);
            *reinterpret_cast<uint4 *>(dst + 16 * k + 8) = make_uint4(a[4], a[5], a[6], a[7]);
        }
    }
    if (p.lse && d0 == 0)
        p.lse[tok * p.q_heads + head] = l == 0.f ? -INFINITY : 0.69314718056f * (m + log2f(l));
}

// kv4_decode.cu
int kv4_decode_ctas();
size_t kv4_decode_part_floats(int head_dim);
// rows: the most rows (new tokens * group) of a sequence, max_units: the most
// units in all, as far as known (0: not known).
uw_status launch_kv4_decode(const AttnParams &p, int head_dim, int64_t rows, int64_t max_units, cudaStream_t st);
// kv4_prefill.cu
int kv4_prefill_ctas();
size_t kv4_prefill_part_floats(int head_dim);
uw_status launch_kv4_prefill(const AttnParams &p, int head_dim, cudaStream_t st);

}  // namespace uw
