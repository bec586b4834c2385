// page_plan.cu -- block tables, slot maps and batch offsets from request
// lengths, on the GPU.
//
// Row s of the block table holds held_s = ceil(held_len_s / P) pages; after
// the step it must hold need_s = ceil(kv_len_s / P).  Rows that shrink (a
// finished or rolled-back request) push their pages past need_s on the stack
// of free pages, in the order of (row, column); rows that grow then take pages
// from its top, in the same order.  With exclusive prefix sums g_s of the pages
// taken and b_s of the pages given back, F the stack's height and R = sum of
// the pages given back, column held_s + j of row s gets entry
// F + R - 1 - (g_s + j) of the stack: below F that is free_pages, from F on the
// (entry - F)-th page given back, found by a search in b.  So every column is
// computed on its own and nothing is read that this launch writes.  If the
// pages do not suffice no page moves and every slot is -1.
//
// A scan over the sequences in one CTA, then one launch over tokens and
// columns.  Bound by latency: a step's whole output is tens of bytes a sequence
// and 8 bytes a token.
#include "dsa_kernels.cuh"

namespace dsa {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;

// Scratch the scan leaves for the fill.
struct PlanScratch {
    int64_t* totals;      // F, pages taken, pages given back, enough (0 / 1)
    int64_t* taken_off;   // [n_seq + 1] exclusive prefix sums
    int64_t* back_off;    // [n_seq + 1]
};

struct SeqPages {
    int64_t kv, q, held, need;
};

// Lengths of sequence s in pages; a row whose lengths make no sense is
// reported and counts as empty.
__device__ __forceinline__ SeqPages seq_pages(const PagePlanArgs& a, int64_t s, int32_t* err) {
    const int64_t h = a.held_len[s], kv = a.kv_len[s], q = a.q_len[s];
    const int64_t cap = a.pg.table_ld << a.pg.shift;
    SeqPages p{0, 0, 0, 0};
    if (h < 0 || kv < 0 || q < 0 || q > kv || h > cap || kv > cap) {
        record_error(err, kDevBadBatch, (int32_t)s, /*where=*/30);
        return p;
    }
    const int64_t round = a.pg.page_rows - 1;
    p.kv = kv;
    p.q = q;
    p.held = (h + round) >> a.pg.shift;
    p.need = (kv + round) >> a.pg.shift;
    return p;
}

// Inclusive prefix sums over the CTA of four values per thread.
__device__ __forceinline__ void block_scan4(int64_t (&v)[4], int64_t (*warp_tot)[4]) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t o = __shfl_up_sync(0xffffffffu, v[k], d);
            if (lane >= d) v[k] += o;
        }
    }
    if (lane == 31) {
#pragma unroll
        for (int k = 0; k < 4; ++k) warp_tot[wid][k] = v[k];
    }
    __syncthreads();
    if (wid == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            int64_t t = warp_tot[lane][k];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, t, d);
                if (lane >= d) t += o;
            }
            warp_tot[lane][k] = t;
        }
    }
    __syncthreads();
    if (wid > 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] += warp_tot[wid - 1][k];
    }
}

__global__ void __launch_bounds__(kScanThreads)
page_plan_scan(PagePlanArgs a, PlanScratch sc, int32_t* err) {
    __shared__ int64_t warp_tot[kScanThreads / 32][4];
    int64_t carry[4] = {0, 0, 0, 0};
    if (threadIdx.x == 0) {
        a.row_off[0] = 0;
        a.q_off[0] = 0;
        sc.taken_off[0] = 0;
        sc.back_off[0] = 0;
    }
    for (int64_t s0 = 0; s0 < a.n_seq; s0 += kScanThreads) {
        const int64_t s = s0 + threadIdx.x;
        SeqPages p{0, 0, 0, 0};
        if (s < a.n_seq) p = seq_pages(a, s, err);
        int64_t v[4] = {p.kv, p.q, p.need > p.held ? p.need - p.held : 0,
                        p.held > p.need ? p.held - p.need : 0};
        block_scan4(v, warp_tot);
        if (s < a.n_seq) {
            a.row_off[s + 1] = carry[0] + v[0];
            a.q_off[s + 1] = carry[1] + v[1];
            sc.taken_off[s + 1] = carry[2] + v[2];
            sc.back_off[s + 1] = carry[3] + v[3];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) carry[k] += warp_tot[kScanThreads / 32 - 1][k];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        int64_t f = *a.n_free_in;
        if (f < 0 || f > a.pg.n_pages) {
            record_error(err, kDevBadBatch, -1, /*where=*/30);
            f = 0;
        }
        // tokens the slot map has no room for, a stack higher than its array
        if (carry[1] > a.max_new) record_error(err, kDevBadBatch, -2, /*where=*/30);
        const bool fits = f + carry[3] <= a.pg.n_pages;
        if (!fits) record_error(err, kDevBadBatch, -3, /*where=*/30);
        const bool enough = fits && carry[2] <= f + carry[3];
        if (fits && !enough)
            record_error(err, kDevNoPages, (int32_t)(carry[2] - f - carry[3]), /*where=*/30);
        sc.totals[0] = f;
        sc.totals[1] = carry[2];
        sc.totals[2] = carry[3];
        sc.totals[3] = enough ? 1 : 0;
        *a.n_free_out = (int32_t)(enough ? f + carry[3] - carry[2] : f);
    }
}

// Last s in [0, n) with off[s] <= x (off[0] <= x).
__device__ __forceinline__ int64_t last_at_most(const int64_t* off, int64_t n, int64_t x) {
    int64_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (off[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Entry `at` of the stack once the step's pages are given back.
__device__ __forceinline__ int32_t stack_entry(const PagePlanArgs& a, const PlanScratch& sc,
                                               int64_t F, int64_t at) {
    if (at < F) return a.free_pages[at];
    const int64_t r = at - F;
    const int64_t s = last_at_most(sc.back_off, a.n_seq, r);
    const int64_t need = (a.kv_len[s] + a.pg.page_rows - 1) >> a.pg.shift;
    return a.block_table[s * a.pg.table_ld + need + (r - sc.back_off[s])];
}

// Blocks below seq_ctas: a warp per sequence writes the columns it takes, and
// the free entries its pages given back end up as.  The others: a thread per
// slot.
__global__ void __launch_bounds__(kFillThreads)
page_plan_fill(PagePlanArgs a, PlanScratch sc, int32_t seq_ctas, int32_t* err) {
    const int64_t F = sc.totals[0], A = sc.totals[1], R = sc.totals[2];
    const bool enough = sc.totals[3] != 0;
    if ((int32_t)blockIdx.x < seq_ctas) {
        const int64_t s = (int64_t)blockIdx.x * (kFillThreads / 32) + (threadIdx.x >> 5);
        const int lane = threadIdx.x & 31;
        if (s >= a.n_seq || !enough) return;
        const int64_t g0 = sc.taken_off[s], g1 = sc.taken_off[s + 1];
        const int64_t b0 = sc.back_off[s], b1 = sc.back_off[s + 1];
        const int64_t held = (a.held_len[s] + a.pg.page_rows - 1) >> a.pg.shift;
        int32_t* row = a.block_table + s * a.pg.table_ld;
        for (int64_t j = lane; j < g1 - g0; j += 32)
            row[held + j] = stack_entry(a, sc, F, F + R - 1 - (g0 + j));
        const int64_t need = (a.kv_len[s] + a.pg.page_rows - 1) >> a.pg.shift;
        for (int64_t j = lane; j < b1 - b0 && F + b0 + j < F + R - A; j += 32)
            a.free_pages[F + b0 + j] = row[need + j];
        return;
    }
    const int64_t i = (int64_t)(blockIdx.x - seq_ctas) * kFillThreads + threadIdx.x;
    if (i >= a.max_new) return;
    int64_t slot = -1;
    if (enough && i < a.q_off[a.n_seq]) {
        const int64_t s = last_at_most(a.q_off, a.n_seq, i);
        const int64_t kv = a.row_off[s + 1] - a.row_off[s];
        const int64_t pos = kv - (a.q_off[s + 1] - a.q_off[s]) + (i - a.q_off[s]);
        const int64_t c = pos >> a.pg.shift;
        const int64_t held = (a.held_len[s] + a.pg.page_rows - 1) >> a.pg.shift;
        const int32_t page =
            c < held ? a.block_table[s * a.pg.table_ld + c]
                     : stack_entry(a, sc, F, F + R - 1 - (sc.taken_off[s] + (c - held)));
        if (page >= 0 && page < a.pg.n_pages)
            slot = ((int64_t)page << a.pg.shift) + (pos & (a.pg.page_rows - 1));
        else
            record_error(err, kDevBadIndex, (int32_t)s, /*where=*/31);
    }
    a.slots[i] = slot;
}

PlanScratch carve(void* scratch, int64_t n_seq) {
    int64_t* p = static_cast<int64_t*>(scratch);
    return PlanScratch{p, p + 4, p + 4 + n_seq + 1};
}

}  // namespace

size_t page_plan_scratch_bytes(int64_t n_seq) { return (size_t)(4 + 2 * (n_seq + 1)) * sizeof(int64_t); }

int32_t page_plan_launches() { return 2; }

cudaError_t launch_page_plan(const PagePlanArgs& a, void* scratch, int32_t* err, cudaStream_t st) {
    const PlanScratch sc = carve(scratch, a.n_seq);
    cudaError_t e = launch_plain(page_plan_scan, dim3(1), dim3(kScanThreads), 0, st, a, sc, err);
    if (e != cudaSuccess) return e;
    const int64_t seq_ctas = (a.n_seq + kFillThreads / 32 - 1) / (kFillThreads / 32);
    const int64_t tok_ctas = (a.max_new + kFillThreads - 1) / kFillThreads;
    if (seq_ctas + tok_ctas == 0) return cudaSuccess;
    return launch_plain(page_plan_fill, dim3((unsigned)(seq_ctas + tok_ctas)), dim3(kFillThreads), 0,
                        st, a, sc, (int32_t)seq_ctas, err);
}

}  // namespace dsa
