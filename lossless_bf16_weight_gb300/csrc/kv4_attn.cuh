// What the attention kernels over the 4-bit paged cache share: their parameters
// (attn_work.cuh has the rest).
#pragma once
#include "attn_work.cuh"

namespace uw {

__device__ __forceinline__ Seq seq_of(const Kv4View &v, int s) { return kv4_seq(v, s); }

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
