// paged_mla.cu -- absorbed-MLA attention over the paged 8-bit cache, CUDA-core
// path (float32 queries), and the launch plan of both paths.
//
// For one query with absorbed query q[h, :] and rows J (its selection, or every
// visible row), a row being its codes times its page's power-of-two scales:
//     z[h,j] = scale * q[h,:] . row_j,  p = softmax_j(z),
//     out[h,c] = sum_j p[h,j] row_j[c] over the 512 latent columns
// ("GLM 5.2 in one C file", "Attention: Multi head Latent Attention With a Tiny
// KV Cache"; "GLM-5.x (glm-dsa, glm5next)", "The block").
//
// A CTA takes 16 heads and a range of one query's rows, 16 at a time: the rows
// are widened to float in shared memory, and each of four warps has four heads --
// a lane forms the logits of two rows and four heads over a quarter of the
// columns, the warp folds the tile into its running maxima and sums by shuffles,
// and each lane accumulates 16 of the 512 outputs of its four heads.  Bound by
// shared-memory reads, so a float4 read is used for 16 multiply-adds and more
// (ten queries of 2,048 rows: 257 us with a half warp to a head and four
// multiply-adds a read, 169 us so, 131 us with the splits below); small float32 steps are bound by latency,
// which is why the heads are spread over CTAs (one query of 256 rows: 27 us with
// all 64 heads in a CTA and the softmax through shared memory, 13.5 us so).  Rows whose index or
// page is out of range are zero and take no weight.  Splits of a query are
// combined by the log-sum-exp merge.
#include <math.h>

#include "dsa_kernels.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 64;
constexpr int kGroup = 16;                       // heads of a CTA
constexpr int kWarpHeads = 4;                    // of a warp
constexpr int kTile = 16;                        // rows per tile
constexpr int kLatent = kLatentCols;

template <int W>
struct Smem {
    static constexpr int kStride = W + 4;        // floats: eight rows' float4s on distinct banks
    static constexpr size_t kRows = kTile * (2 * sizeof(int64_t));
    static constexpr size_t kQ = (size_t)kGroup * kStride * sizeof(float);
    static constexpr size_t kR = (size_t)kTile * kStride * sizeof(float);
    static constexpr size_t kP = (size_t)kGroup * kTile * sizeof(float);
    static constexpr size_t kTotal = kRows + kQ + kR + kP;
};

__device__ __forceinline__ void fma4(float4& a, const float4& x, const float4& y) {
    a.x = fmaf(x.x, y.x, a.x);
    a.y = fmaf(x.y, y.y, a.y);
    a.z = fmaf(x.z, y.z, a.z);
    a.w = fmaf(x.w, y.w, a.w);
}

template <int FMT, int W>
__global__ void __launch_bounds__(kThreads, 3)
paged_mla_simt(BatchDev b, PagedCache pc, float scale, const float* __restrict__ q_abs,
               const int32_t* __restrict__ idx, const int32_t* __restrict__ n_sel,
               int64_t idx_width, int32_t rows_per_split, int32_t n_split,
               float* __restrict__ out, float* __restrict__ lse, float* __restrict__ part_o,
               float* __restrict__ part_ml, int32_t* err) {
    using S = Smem<W>;
    constexpr int kParts = W > kLatent ? 2 : 1;
    constexpr int kRowVecs = W / 16;                   // 16-byte vectors of codes
    extern __shared__ __align__(16) unsigned char smem[];
    int64_t* row_at = reinterpret_cast<int64_t*>(smem);              // pool row, -1: none
    float2* row_scale = reinterpret_cast<float2*>(row_at + kTile);
    float* Qs = reinterpret_cast<float*>(smem + S::kRows);
    float* Rs = reinterpret_cast<float*>(smem + S::kRows + S::kQ);
    float* Ps = reinterpret_cast<float*>(smem + S::kRows + S::kQ + S::kR);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int tid = threadIdx.x;
    const int64_t q = blockIdx.y;
    const int split = blockIdx.x, h0 = kGroup * blockIdx.z;
    const int warp = tid >> 5, lane = tid & 31;
    const int hw = kWarpHeads * warp;                  // this warp's first head of the group
    const int rg = lane & 7, kq = lane >> 3;           // this lane's rows rg, rg + 8; its quarter of the columns
    const int64_t part = q * n_split + split;
    QueryInfo qi;
    if (!query_info(b, q, qi, err, /*where=*/33)) {
        if (n_split > 1 && tid < kGroup) {             // no weight in the merge
            part_ml[(part * kHeads + h0 + tid) * 2 + 0] = -INFINITY;
            part_ml[(part * kHeads + h0 + tid) * 2 + 1] = 0.f;
        }
        return;
    }
    int64_t ns = idx == nullptr ? qi.L : n_sel[q];
    if (idx != nullptr) ns = ns < 0 ? 0 : (ns > idx_width ? idx_width : ns);
    const int64_t j_begin = (int64_t)split * rows_per_split;
    const int64_t j_end = j_begin + rows_per_split < ns ? j_begin + rows_per_split : ns;

    const float* qsrc = q_abs + (q * kHeads + h0) * (int64_t)W;
    for (int v = tid; v < kGroup * (W / 4); v += kThreads) {
        const int r = v / (W / 4), c = (v % (W / 4)) * 4;
        *reinterpret_cast<float4*>(Qs + r * S::kStride + c) =
            __ldg(reinterpret_cast<const float4*>(qsrc + (int64_t)r * W + c));
    }

    bool rows = false;                                 // any that exists
    float m[kWarpHeads], l[kWarpHeads];                // the same in all lanes of the warp
    float4 o[kWarpHeads][kLatent / 128];               // columns 4 lane + 128 i
#pragma unroll
    for (int k = 0; k < kWarpHeads; ++k) {
        m[k] = -INFINITY;
        l[k] = 0.f;
#pragma unroll
        for (int i = 0; i < kLatent / 128; ++i) o[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    for (int64_t t0 = j_begin; t0 < j_end; t0 += kTile) {
        const int nrows = (int)(j_end - t0 < kTile ? j_end - t0 : kTile);
        if (tid < kTile) {
            int64_t at = -1;
            float2 f = make_float2(0.f, 0.f);
            if (tid < nrows) {
                const int32_t r = idx == nullptr ? (int32_t)(t0 + tid) : idx[q * idx_width + t0 + tid];
                const int32_t page = r >= 0 && r < qi.L ? page_of(pc.pg, pc.block_table, qi.seq, r) : -1;
                if (page >= 0) {
                    at = ((int64_t)page << pc.pg.shift) + (r & (pc.pg.page_rows - 1));
                    f.x = e8m0(pc.scales[(int64_t)page * kParts]);
                    if (kParts == 2) f.y = e8m0(pc.scales[(int64_t)page * kParts + 1]);
                } else {
                    record_error(err, kDevBadIndex, (int32_t)q, /*where=*/33);
                }
            }
            row_at[tid] = at;
            row_scale[tid] = f;
        }
        __syncthreads();
        for (int v = tid; v < kTile * kRowVecs; v += kThreads) {
            const int r = v / kRowVecs, c = (v % kRowVecs) * 16;
            const int64_t at = row_at[r];
            uint4 w = make_uint4(0, 0, 0, 0);
            if (at >= 0) w = __ldg(reinterpret_cast<const uint4*>(pc.codes + at * W + c));
            const float f = at < 0 ? 0.f : (c < kLatent ? row_scale[r].x : row_scale[r].y);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float x[4];
                widen_codes<FMT>(u[k], x);
                *reinterpret_cast<float4*>(Rs + r * S::kStride + c + 4 * k) =
                    make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
            }
        }
        __syncthreads();
        rows |= row_at[rg] >= 0 || row_at[rg + 8] >= 0;
        // the logits of two rows and four heads over a quarter of the columns
        float z[kWarpHeads][2];
        {
            float4 acc[kWarpHeads][2];
#pragma unroll
            for (int k = 0; k < kWarpHeads; ++k) acc[k][0] = acc[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int c = 4 * kq; c < W; c += 16) {
                const float4 ra = *reinterpret_cast<const float4*>(Rs + rg * S::kStride + c);
                const float4 rb = *reinterpret_cast<const float4*>(Rs + (rg + 8) * S::kStride + c);
#pragma unroll
                for (int k = 0; k < kWarpHeads; ++k) {
                    const float4 q4 = *reinterpret_cast<const float4*>(Qs + (hw + k) * S::kStride + c);
                    fma4(acc[k][0], q4, ra);
                    fma4(acc[k][1], q4, rb);
                }
            }
#pragma unroll
            for (int k = 0; k < kWarpHeads; ++k) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = (acc[k][i].x + acc[k][i].y) + (acc[k][i].z + acc[k][i].w);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    z[k][i] = row_at[rg + 8 * i] >= 0 ? x * scale : -INFINITY;
                }
            }
        }
        float alpha[kWarpHeads];
#pragma unroll
        for (int k = 0; k < kWarpHeads; ++k) {
            float mx = fmaxf(z[k][0], z[k][1]);
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float m_new = fmaxf(m[k], mx);
            // no maximum yet: rows without weight, or a NaN logit to pass on
            const float p0 = z[k][0] == -INFINITY ? 0.f : expf(z[k][0] - m_new);
            const float p1 = z[k][1] == -INFINITY ? 0.f : expf(z[k][1] - m_new);
            alpha[k] = m_new == -INFINITY ? 1.f : expf(m[k] - m_new);
            float sum = p0 + p1;
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l[k] = l[k] * alpha[k] + sum;
            m[k] = m_new;
            if (kq == k) {                             // [row][head], read by this warp alone
                Ps[(warp * kTile + rg) * kWarpHeads + k] = p0;
                Ps[(warp * kTile + rg + 8) * kWarpHeads + k] = p1;
            }
#pragma unroll
            for (int i = 0; i < kLatent / 128; ++i) {
                o[k][i].x *= alpha[k]; o[k][i].y *= alpha[k]; o[k][i].z *= alpha[k]; o[k][i].w *= alpha[k];
            }
        }
        __syncwarp();
#pragma unroll 2
        for (int r = 0; r < nrows; ++r) {
            const float4 w = *reinterpret_cast<const float4*>(Ps + (warp * kTile + r) * kWarpHeads);
            const float wk[kWarpHeads] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < kLatent / 128; ++i) {
                const float4 r4 = *reinterpret_cast<const float4*>(Rs + r * S::kStride + 4 * lane + 128 * i);
#pragma unroll
                for (int k = 0; k < kWarpHeads; ++k)
                    fma4(o[k][i], make_float4(wk[k], wk[k], wk[k], wk[k]), r4);
            }
        }
        __syncthreads();
    }

    const bool last = n_split == 1;
    rows = __any_sync(0xffffffffu, rows);
#pragma unroll
    for (int k = 0; k < kWarpHeads; ++k) {
        const int h = h0 + hw + k;
        // rows whose logits are all -inf: NaN, as of any softmax of those, unless
        // another split has more (m = -inf, l = 1 for the merge)
        const bool lost = rows && l[k] == 0.f;
        const float inv = last ? (l[k] == 0.f ? (lost ? NAN : 0.f) : 1.f / l[k]) : 1.f;
        float* dst = (last ? out + (q * kHeads + h) * (int64_t)kLatent
                           : part_o + (part * kHeads + h) * (int64_t)kLatent) + 4 * lane;
#pragma unroll
        for (int i = 0; i < kLatent / 128; ++i)
            *reinterpret_cast<float4*>(dst + 128 * i) =
                make_float4(o[k][i].x * inv, o[k][i].y * inv, o[k][i].z * inv, o[k][i].w * inv);
        if (lane == 0) {
            if (last) {
                if (lse != nullptr) lse[q * kHeads + h] = l[k] != 0.f ? m[k] + logf(l[k]) : lost ? NAN : -INFINITY;
            } else {
                // rows whose logits are all NaN: a split with weight
                part_ml[(part * kHeads + h) * 2 + 0] = m[k] == -INFINITY && l[k] != 0.f ? 0.f : m[k];
                part_ml[(part * kHeads + h) * 2 + 1] = lost ? 1.f : l[k];
            }
        }
    }
}

// Rows a query attends over at most, and the rows that size its splits: the
// k-pool tail (fewer than kpool rows past the selected pools' top_k) sizes
// none, it spills into one more, short split.
void paged_rows(const Shape& sh, const BatchDev& b, int64_t* main_rows, int64_t* max_rows) {
    *max_rows = *main_rows = b.max_kv_len;
    if (!(b.flags & DSA_FLAG_DENSE) && sh.index_row_width() < *max_rows) {
        *max_rows = sh.index_row_width();
        *main_rows = sh.top_k;
    }
    if (*max_rows < 1) *max_rows = 1;
    if (*main_rows < 1 || *main_rows > *max_rows) *main_rows = *max_rows;
}

// CUDA-core splits: with the four head groups at most the CTAs that are resident
// at once, three a multiprocessor, and at least one tile each.  (Four a
// multiprocessor, rounded up: ten queries of 2,048 rows 169 us, one query 36.7 us;
// so 131 and 25.7 us.)
void plan_splits_simt(int32_t n_q, int64_t max_rows, int32_t* rows_per_split, int32_t* n_split) {
    const int64_t target = 3 * (int64_t)sm_count() / (kHeads / kGroup);
    const int64_t tiles = (max_rows + kTile - 1) / kTile;
    int64_t splits = target / n_q;
    if (splits > tiles) splits = tiles;
    if (splits < 1) splits = 1;
    const int64_t rps = (tiles + splits - 1) / splits * kTile;
    *rows_per_split = (int32_t)rps;
    *n_split = (int32_t)((max_rows + rps - 1) / rps);
}

template <int FMT, int W>
cudaError_t launch_t(const Shape& sh, const BatchDev& b, const PagedCache& pc, const void* q_abs,
                     const int32_t* idx, const int32_t* n_sel, float* out, float* lse,
                     float* part_o, float* part_ml, int32_t rps, int32_t n_split, int32_t* err,
                     cudaStream_t st) {
    using S = Smem<W>;
    auto kern = paged_mla_simt<FMT, W>;
    cudaError_t e = ensure_dyn_smem((const void*)kern, (int)S::kTotal);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)n_split, (unsigned)b.n_q, kHeads / kGroup), dim3(kThreads),
                   S::kTotal, st, b, pc, sh.scale, static_cast<const float*>(q_abs), idx, n_sel,
                   sh.index_row_width(), rps, n_split, out, lse, part_o, part_ml, err);
    if (e != cudaSuccess || n_split == 1) return e;
    return launch_merge_splits(b.n_q, n_split, part_o, part_ml, out, lse, st, /*nan_lse=*/true);
}

}  // namespace

// Rows that a tensor-core CTA takes at a time; the most rows that are planned by
// whole tiles.
constexpr int64_t kPlanTile = 64;
constexpr int64_t kMostPlanned = 0x7fffffff / kPlanTile * kPlanTile;

// Splits by the rows of all sequences together (below): one query to a sequence, and
// at least half of the multiprocessors to spare.
bool decode_batch_plan(const BatchDev& b) {
    return b.n_q == b.n_seq && sm_count() - b.n_q >= sm_count() / 2;
}

void plan_paged_splits(const Shape& sh, const BatchDev& b, int32_t* rows_per_split,
                       int32_t* n_split) {
    int64_t main_rows, max_rows;
    paged_rows(sh, b, &main_rows, &max_rows);
    const int32_t n_q = b.n_q > 0 ? b.n_q : 1;
    // Whole tiles of the longest bounds would pass 32 bits: the plan is made for less,
    // and its one split, or one more, takes the rest.
    const int64_t planned = max_rows < kMostPlanned ? max_rows : kMostPlanned;
    if (sh.dtype != DSA_BF16)
        plan_splits_simt(n_q, planned, rows_per_split, n_split);
    else
        plan_attention_splits_tc(n_q, main_rows < planned ? main_rows : planned, planned,
                                 rows_per_split, n_split);
    if (planned < max_rows) {
        if (*n_split == 1) *rows_per_split = (int32_t)max_rows;
        *n_split = (int32_t)((max_rows + *rows_per_split - 1) / *rows_per_split);
    }
    if (sh.dtype != DSA_BF16) return;
    // With one query to a sequence the batch's rows bound those of all queries
    // together: splits of r rows then give at most rows / r + n_q CTAs with work,
    // however the lengths differ (the others end at once), so r is chosen for one
    // wave of those instead of one wave of the longest sequence's.  Eight dense
    // sequences of 20,000 to 100,003 rows: 230 us with the longest's, 174 us so.
    // The partials grow with the longest sequence's splits: up to four waves' of them.
    if (!decode_batch_plan(b) || *n_split <= 2) return;
    const int64_t sms = sm_count(), spare = sms - n_q;
    const int64_t tiles = (b.total_rows + kPlanTile - 1) / kPlanTile;
    int64_t rps = (tiles + spare - 1) / spare * kPlanTile;
    if (rps < 2 * kPlanTile) rps = 2 * kPlanTile;
    const int64_t fewest = (max_rows * n_q + 4 * sms - 1) / (4 * sms);
    if (rps < fewest) rps = (fewest + kPlanTile - 1) / kPlanTile * kPlanTile;
    if (rps >= *rows_per_split) return;
    *rows_per_split = (int32_t)rps;
    *n_split = (int32_t)((max_rows + rps - 1) / rps);
}

// Partials for the most splits that any batch of these queries with fewer rows could
// be given, so that a workspace sized for a program's bounds serves all its batches.
size_t paged_mla_scratch_bytes(const Shape& sh, const BatchDev& b) {
    int64_t main_rows, max_rows;
    paged_rows(sh, b, &main_rows, &max_rows);
    const int64_t n_q = b.n_q > 0 ? b.n_q : 1, sms = sm_count();
    const bool tail = main_rows < max_rows;
    int64_t splits, least;                           // and the fewest rows of one but the last
    if (sh.dtype != DSA_BF16) {
        splits = 3 * sms / (kHeads / kGroup) / n_q;
        least = kTile;
    } else {
        splits = decode_batch_plan(b) ? (4 * sms + n_q - 1) / n_q : sms / n_q;
        least = n_q == 1 ? kPlanTile : 2 * kPlanTile;
    }
    const int64_t whole = (max_rows + least - 1) / least;
    if (splits > whole) splits = whole;
    if (splits < 1) splits = 1;
    if (max_rows > kMostPlanned || (sh.dtype == DSA_BF16 && tail)) ++splits;
    if (splits == 1) return 0;
    return (size_t)n_q * splits * kHeads * (kLatent + 2) * sizeof(float);
}

int32_t paged_mla_launches(const Shape& sh, const BatchDev& b) {
    int32_t rps, n_split;
    plan_paged_splits(sh, b, &rps, &n_split);
    // two tensor-core splits merge inside their launch
    return n_split > (sh.dtype == DSA_BF16 ? 2 : 1) ? 2 : 1;
}

cudaError_t launch_paged_mla(const Shape& sh, const BatchDev& b, const PagedCache& pc,
                             const void* q_abs, const int32_t* idx, const int32_t* n_sel,
                             float* out, float* lse, void* scratch, size_t scratch_bytes,
                             int32_t* err, cudaStream_t st) {
    if (b.n_q == 0) return cudaSuccess;
    int32_t rps, n_split;
    plan_paged_splits(sh, b, &rps, &n_split);
    float* part_o = nullptr;
    float* part_ml = nullptr;
    if (n_split > 1) {
        const size_t parts = (size_t)b.n_q * n_split * kHeads;
        if (scratch == nullptr || scratch_bytes < parts * (kLatent + 2) * sizeof(float))
            return cudaErrorInvalidValue;
        part_o = static_cast<float*>(scratch);
        part_ml = part_o + parts * kLatent;
    }
    if (sh.dtype == DSA_BF16)
        return launch_paged_mla_tc(sh, b, pc, q_abs, idx, n_sel, out, lse, part_o, part_ml, rps,
                                   n_split, err, st);
    const bool wide = sh.width() == 576;
    auto f = pc.pg.format == DSA_CACHE_E4M3 ? (wide ? launch_t<DSA_CACHE_E4M3, 576> : launch_t<DSA_CACHE_E4M3, 512>)
                                            : (wide ? launch_t<DSA_CACHE_S8, 576> : launch_t<DSA_CACHE_S8, 512>);
    return f(sh, b, pc, q_abs, idx, n_sel, out, lse, part_o, part_ml, rps, n_split, err, st);
}

}  // namespace dsa
