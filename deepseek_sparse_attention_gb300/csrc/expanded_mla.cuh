// expanded_mla.cuh -- what the kernels of the expanded latent attention share:
// the units of work and where their results go.
#pragma once

#include "dsa_kernels.cuh"

namespace dsa {

// The operands, as the kernels take them.
struct ExpandedArgs {
    const void *q, *k_nope, *rows, *v;
    void* out;
    float* lse;
    float *part_o, *part_ml;       // partial sums of splits (float32), where there are several
    int32_t heads, nope, rope, v_dim, kv_lora, width;
    int32_t n_split;
    float scale;
    BatchDev b;
    int32_t* err;
};

// A tile of up to `bq` queries of one sequence and the key tiles of one split.
struct ExpandedTile {
    int64_t q0;                    // first query of the tile
    int64_t row0;                  // first cache row of the sequence
    int64_t first;                 // rows that the tile's first query sees
    int32_t n_q;                   // its queries
    int32_t kt0, kt1;              // key tiles of the split
};

// Tiles have slots: sequence s has the slots from start(s) = q_off[s] / bq + min(s,
// q_off[s]) on, up to start(s + 1).  That is room for its ceil(q_len / bq) tiles:
// where q_len > 0 the first term grows by q_len / bq rounded down at least and the
// second by one at least.  So a slot finds its sequence by a search over the offsets,
// nothing is planned ahead, and idle sequences, of which a batch may have many, add no
// slots beyond the queries' number.  Slots left over have no tile.
__host__ __device__ inline int64_t expanded_slots(int64_t n_q, int64_t n_seq, int bq) {
    return n_q / bq + (n_seq < n_q ? n_seq : n_q);
}
__host__ __device__ inline int64_t expanded_start(const BatchDev& b, int32_t s, int bq) {
    const int64_t q = b.q_off[s];
    return q / bq + (s < q ? s : q);
}

// Whether sequence s lies within the bounds that the host gave, and whether the batch's ends do.
__host__ __device__ inline bool expanded_within(const BatchDev& b, int64_t q0, int64_t q1, int64_t r0, int64_t r1) {
    return q0 >= 0 && q1 >= q0 && q1 <= b.n_q && q1 - q0 <= b.max_q_len && r0 >= 0 && r1 >= r0 && r1 <= b.total_rows &&
           r1 - r0 <= b.max_kv_len && q1 - q0 <= r1 - r0;
}
__host__ __device__ inline bool expanded_sound(const BatchDev& b, int32_t s) {
    return expanded_within(b, b.q_off[s], b.q_off[s + 1], b.row_off[s], b.row_off[s + 1]);
}
__host__ __device__ inline bool expanded_ends_sound(const BatchDev& b) {
    return b.q_off[0] == 0 && b.q_off[b.n_seq] == b.n_q;
}
// Records sequences at, at + step, ... that are not.  The search for a slot's sequence need not
// come to them: starts in disorder may hide one, and idle ones may have no slot.
__device__ __forceinline__ void expanded_check(const BatchDev& b, int64_t at, int64_t step, int32_t* err, int32_t where) {
    if (at == 0 && !expanded_ends_sound(b)) record_error(err, kDevBadBatch, b.n_seq, where);
    for (; at < b.n_seq; at += step)
        if (!expanded_sound(b, (int32_t)at)) record_error(err, kDevBadBatch, (int32_t)at, where);
}

// False if the slot has no tile, or its sequence is not sound.
__host__ __device__ inline bool expanded_tile(const BatchDev& b, int64_t slot, int32_t split, int32_t n_split, int bq,
                                              int bk, ExpandedTile& t) {
    int32_t lo = 0, hi = b.n_seq - 1;
    while (lo < hi) {                                    // last s whose slots start at or before this one
        const int32_t mid = lo + (hi - lo + 1) / 2;
        if (expanded_start(b, mid, bq) <= slot) lo = mid; else hi = mid - 1;
    }
    const int64_t q0 = b.q_off[lo], q1 = b.q_off[lo + 1], r0 = b.row_off[lo], r1 = b.row_off[lo + 1];
    if (!expanded_within(b, q0, q1, r0, r1)) return false;
    const int64_t q_len = q1 - q0, kv_len = r1 - r0;
    const int64_t at = slot - (q0 / bq + (lo < q0 ? lo : q0));
    if (at < 0 || at * bq >= q_len) return false;
    t.q0 = q0 + at * bq;
    t.row0 = r0;
    t.n_q = (int32_t)(q_len - at * bq < bq ? q_len - at * bq : bq);
    t.first = kv_len - q_len + 1 + at * bq;
    const int64_t tiles = (t.first + t.n_q - 1 + bk - 1) / bk;   // up to the last query's last row
    t.kt0 = (int32_t)(tiles * split / n_split);
    t.kt1 = (int32_t)(tiles * (split + 1) / n_split);
    return true;
}

// Log2 of a sum of exponentials with maximum m (in log2 units) and sum l to the
// natural logarithm; NaN where every attended logit was -inf (l == 0).
__device__ __forceinline__ float expanded_lse(float m, float l) {
    return l == 0.f ? __int_as_float(0x7fffffff) : (m + log2f(l)) * 0.6931471805599453f;
}

// The tensor-core kernel (expanded_mla_tc.cu), bf16: its tiles.
constexpr int kExpandedTcQ = 256, kExpandedTcK = 128;
cudaError_t launch_expanded_tc(const ExpandedArgs& a, cudaStream_t st);

}  // namespace dsa
