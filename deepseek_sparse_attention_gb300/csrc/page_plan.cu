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
// pages do not suffice, or F is no height the stack can have, no page moves and
// every slot is -1.
//
// A page that two rows name would be pushed while one of them still reads it, or
// twice.  Rows' held pages and free pages that are all different are n_pages at
// most; more of them hold some page twice, and then nothing is given back.
//
// Bound by latency: a step's whole output is tens of bytes a sequence and 8
// bytes a token.  Up to 1,024 sequences are one launch, in which every CTA scans
// them all for itself (24 KB from L2) and keeps the sums in shared memory for its
// searches; more are a scan in one CTA, then a launch over tokens and columns.
#include "dsa_kernels.cuh"

namespace dsa {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kSmallSeqs = 1024;          // sequences of the one-launch plan
constexpr int kSmallThreads = 256;
constexpr int kPer = kSmallSeqs / kSmallThreads;

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

constexpr int kScans = 4;                 // rows, tokens, pages taken, pages given back
constexpr int kSums = 5;                  // and pages held

// What sequence s adds to each.
__device__ __forceinline__ void seq_sums(const SeqPages& p, int64_t (&v)[kScans], uint32_t& held) {
    v[0] += p.kv;
    v[1] += p.q;
    v[2] += p.need > p.held ? p.need - p.held : 0;
    v[3] += p.held > p.need ? p.held - p.need : 0;
    held += (uint32_t)p.held;
}

// Sum over the warp of numbers below 2^43.
__device__ __forceinline__ int64_t warp_sum(uint64_t x) {
    const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)(x & 0xffffu));
    return ((int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)(x >> 16)) << 16) + lo;
}

// Inclusive prefix sums over the CTA of kScans values per thread; their totals, and
// that of `held`, are left in warp_tot[31].
__device__ __forceinline__ void block_scan(int64_t (&v)[kScans], uint32_t held,
                                           int64_t (*warp_tot)[kSums]) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int64_t h = warp_sum(held);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
#pragma unroll
        for (int k = 0; k < kScans; ++k) {
            const int64_t o = __shfl_up_sync(0xffffffffu, v[k], d);
            if (lane >= d) v[k] += o;
        }
    }
    if (lane == 31) {
#pragma unroll
        for (int k = 0; k < kScans; ++k) warp_tot[wid][k] = v[k];
        warp_tot[wid][kScans] = h;
    }
    __syncthreads();
    if (wid == 0) {
        const int64_t all = warp_sum(lane < nw ? warp_tot[lane][kScans] : 0);
#pragma unroll
        for (int k = 0; k < kScans; ++k) {
            int64_t t = lane < nw ? warp_tot[lane][k] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, t, d);
                if (lane >= d) t += o;
            }
            warp_tot[lane][k] = t;
        }
        warp_tot[lane][kScans] = all;
    }
    __syncthreads();
    if (wid > 0) {
#pragma unroll
        for (int k = 0; k < kScans; ++k) v[k] += warp_tot[wid - 1][k];
    }
}

// The stack's height, whether the pages suffice, and the reports of what does
// not fit: tokens beyond the slot map, pages that some rows or the stack name
// twice, too few pages.
struct Verdict {
    int64_t F;                 // 0 for a height that the stack cannot have
    bool enough;               // pages move
    int32_t height;            // n_free_out
};
__device__ __forceinline__ Verdict judge(const PagePlanArgs& a, const int64_t (&sum)[kSums],
                                         bool report, int32_t* err) {
    const int64_t tokens = sum[1], taken = sum[2], back = sum[3], held = sum[4];
    const int32_t given = *a.n_free_in;
    const bool bad_f = given < 0 || given > a.pg.n_pages;
    const int64_t f = bad_f ? 0 : given;
    const bool fits = back == 0 || f + held <= a.pg.n_pages;
    const bool enough = !bad_f && fits && taken <= f + back;
    if (report) {
        if (bad_f) record_error(err, kDevBadBatch, -1, /*where=*/30);
        if (tokens > a.max_new) record_error(err, kDevBadBatch, -2, /*where=*/30);
        if (!fits) record_error(err, kDevBadBatch, -3, /*where=*/30);
        else if (taken > f + back) record_error(err, kDevNoPages, (int32_t)(taken - f - back), /*where=*/30);
    }
    return Verdict{f, enough, enough ? (int32_t)(f + back - taken) : given};
}

__global__ void __launch_bounds__(kScanThreads)
page_plan_scan(PagePlanArgs a, PlanScratch sc, int32_t* err) {
    __shared__ int64_t warp_tot[kScanThreads / 32][kSums];
    int64_t carry[kSums] = {0, 0, 0, 0, 0};
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
        int64_t v[kScans] = {0, 0, 0, 0};
        uint32_t held = 0;
        seq_sums(p, v, held);
        block_scan(v, held, warp_tot);
        if (s < a.n_seq) {
            a.row_off[s + 1] = carry[0] + v[0];
            a.q_off[s + 1] = carry[1] + v[1];
            sc.taken_off[s + 1] = carry[2] + v[2];
            sc.back_off[s + 1] = carry[3] + v[3];
        }
#pragma unroll
        for (int k = 0; k < kSums; ++k) carry[k] += warp_tot[31][k];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const Verdict v = judge(a, carry, true, err);
        sc.totals[0] = v.F;
        sc.totals[1] = carry[2];
        sc.totals[2] = carry[3];
        sc.totals[3] = v.enough ? 1 : 0;
        *a.n_free_out = v.height;
    }
}

// Last s in [0, n) with off[s] <= x (off[0] <= x).
template <typename T>
__device__ __forceinline__ int last_at_most(const T* off, int n, int64_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The plan as its second half sees it: the offsets of the sequences' tokens, of
// the pages they take and of those they give back (exclusive prefix sums, n_seq
// + 1 entries; T: int64 in global memory, int32 page counts in shared memory).
template <typename T>
struct Plan {
    const PagePlanArgs& a;
    const int64_t* q_off;
    const T* taken_off;
    const T* back_off;
    int64_t F, A, R;
    bool enough;

    __device__ int64_t pages(int64_t len) const { return (len + a.pg.page_rows - 1) >> a.pg.shift; }
    // Entry `at` of the stack once the step's pages are given back.
    __device__ int32_t stack_entry(int64_t at) const {
        if (at < F) return a.free_pages[at];
        const int64_t r = at - F;
        const int s = last_at_most(back_off, (int)a.n_seq, r);
        return a.block_table[s * a.pg.table_ld + pages(a.kv_len[s]) + (r - back_off[s])];
    }
    // One warp: the columns that sequence s takes, and the free entries its pages
    // given back end up as.
    __device__ void sequence(int64_t s, int lane) const {
        const int64_t g0 = taken_off[s], g1 = taken_off[s + 1], b0 = back_off[s], b1 = back_off[s + 1];
        int32_t* row = a.block_table + s * a.pg.table_ld;
        if (g1 > g0) {
            const int64_t held = pages(a.held_len[s]);
            for (int64_t j = lane; j < g1 - g0; j += 32) row[held + j] = stack_entry(F + R - 1 - (g0 + j));
        }
        if (b1 > b0) {
            const int64_t need = pages(a.kv_len[s]);
            for (int64_t j = lane; j < b1 - b0 && F + b0 + j < F + R - A; j += 32)
                a.free_pages[F + b0 + j] = row[need + j];
        }
    }
    // The slot of new token i.
    __device__ void token(int64_t i, int32_t* err) const {
        int64_t slot = -1;
        if (enough && i < q_off[a.n_seq]) {
            const int s = last_at_most(q_off, (int)a.n_seq, i);
            const int64_t pos = a.kv_len[s] - a.q_len[s] + (i - q_off[s]), c = pos >> a.pg.shift;
            const int64_t held = pages(a.held_len[s]);
            const int32_t page = c < held ? a.block_table[s * a.pg.table_ld + c]
                                          : stack_entry(F + R - 1 - (taken_off[s] + (c - held)));
            if (page >= 0 && page < a.pg.n_pages)
                slot = ((int64_t)page << a.pg.shift) + (pos & (a.pg.page_rows - 1));
            else
                record_error(err, kDevBadIndex, s, /*where=*/31);
        }
        a.slots[i] = slot;
    }
};

// Blocks below seq_ctas: a warp per sequence.  The others: a thread per slot.
__global__ void __launch_bounds__(kFillThreads)
page_plan_fill(PagePlanArgs a, PlanScratch sc, int32_t seq_ctas, int32_t* err) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Plan<int64_t> p{a, a.q_off, sc.taken_off, sc.back_off, sc.totals[0], sc.totals[1],
                          sc.totals[2], sc.totals[3] != 0};
    if ((int32_t)blockIdx.x < seq_ctas) {
        const int64_t s = (int64_t)blockIdx.x * (kFillThreads / 32) + (threadIdx.x >> 5);
        if (s < a.n_seq && p.enough) p.sequence(s, threadIdx.x & 31);
        return;
    }
    const int64_t i = (int64_t)(blockIdx.x - seq_ctas) * kFillThreads + threadIdx.x;
    if (i < a.max_new) p.token(i, err);
}

// The whole plan of up to kSmallSeqs sequences.  `ticket`: a zeroed word; the
// last CTA to have read n_free_in writes n_free_out (they may be one word) and
// leaves the ticket zero again.  Page counts fit 32 bits here: 2^10 rows of fewer
// than 2^27 entries, less than 2^31 of them in all or the plan does not fit.
__global__ void __launch_bounds__(kSmallThreads)
page_plan_small(PagePlanArgs a, uint32_t* ticket, int32_t* err) {
    __shared__ int64_t warp_tot[32][kSums];
    __shared__ int64_t q_off[kSmallSeqs + 1];
    __shared__ uint32_t taken_off[kSmallSeqs + 1], back_off[kSmallSeqs + 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int n = (int)a.n_seq, first = threadIdx.x * kPer;
    int64_t v[kScans] = {0, 0, 0, 0}, each[kPer][kScans];
    uint32_t held = 0;                                 // four rows of fewer than 2^27 pages
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        SeqPages p{0, 0, 0, 0};
        if (first + k < n) p = seq_pages(a, first + k, err);
        seq_sums(p, v, held);
#pragma unroll
        for (int i = 0; i < kScans; ++i) each[k][i] = v[i];
    }
    const int64_t own[kScans] = {v[0], v[1], v[2], v[3]};
    block_scan(v, held, warp_tot);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int s = first + k;
        if (s >= n) break;
        q_off[s + 1] = v[1] - own[1] + each[k][1];
        taken_off[s + 1] = (uint32_t)(v[2] - own[2] + each[k][2]);
        back_off[s + 1] = (uint32_t)(v[3] - own[3] + each[k][3]);
        if (blockIdx.x == 0) {
            a.row_off[s + 1] = v[0] - own[0] + each[k][0];
            a.q_off[s + 1] = q_off[s + 1];
        }
    }
    if (threadIdx.x == 0) {
        q_off[0] = 0;
        taken_off[0] = back_off[0] = 0;
        if (blockIdx.x == 0) a.row_off[0] = a.q_off[0] = 0;
    }
    const int64_t A = warp_tot[31][2], R = warp_tot[31][3];
    const Verdict verdict = judge(a, warp_tot[31], blockIdx.x == 0 && threadIdx.x == 0, err);
    __syncthreads();                                   // the offsets are in, n_free_in is read
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(ticket, 1u) == gridDim.x - 1) {
            *ticket = 0;
            *a.n_free_out = verdict.height;
        }
    }
    const Plan<uint32_t> p{a, q_off, taken_off, back_off, verdict.F, A, R, verdict.enough};
    const int warps = gridDim.x * (kSmallThreads / 32);
    if (p.enough)
        for (int s = blockIdx.x * (kSmallThreads / 32) + (threadIdx.x >> 5); s < n; s += warps)
            p.sequence(s, threadIdx.x & 31);
    for (int64_t i = (int64_t)blockIdx.x * kSmallThreads + threadIdx.x; i < a.max_new;
         i += (int64_t)gridDim.x * kSmallThreads)
        p.token(i, err);
}

PlanScratch carve(void* scratch, int64_t n_seq) {
    int64_t* p = static_cast<int64_t*>(scratch);
    return PlanScratch{p, p + 4, p + 4 + n_seq + 1};
}

}  // namespace

size_t page_plan_scratch_bytes(int64_t n_seq) {
    return n_seq <= kSmallSeqs ? 0 : (size_t)(4 + 2 * (n_seq + 1)) * sizeof(int64_t);
}

int32_t page_plan_launches(int64_t n_seq) { return n_seq <= kSmallSeqs ? 1 : 2; }

cudaError_t launch_page_plan(const PagePlanArgs& a, void* scratch, uint32_t* ticket, int32_t* err,
                             cudaStream_t st) {
    const int64_t seq_ctas = (a.n_seq + kFillThreads / 32 - 1) / (kFillThreads / 32);
    const int64_t tok_ctas = (a.max_new + kFillThreads - 1) / kFillThreads;
    if (a.n_seq <= kSmallSeqs) {
        // a CTA for every eight sequences or 256 tokens, up to four a multiprocessor
        int64_t ctas = seq_ctas > tok_ctas ? seq_ctas : tok_ctas;
        if (ctas > 4 * (int64_t)sm_count()) ctas = 4 * (int64_t)sm_count();
        return launch_pdl(page_plan_small, dim3((unsigned)(ctas > 0 ? ctas : 1)), dim3(kSmallThreads), 0,
                          st, a, ticket, err);
    }
    const PlanScratch sc = carve(scratch, a.n_seq);
    cudaError_t e = launch_plain(page_plan_scan, dim3(1), dim3(kScanThreads), 0, st, a, sc, err);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_plan_fill, dim3((unsigned)(seq_ctas + tok_ctas)), dim3(kFillThreads), 0, st,
                      a, sc, (int32_t)seq_ctas, err);
}

}  // namespace dsa
