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
// A CTA takes a range of one query's rows, 16 at a time: the rows are widened
// to float in shared memory, the 64 x 16 logits formed against the staged
// query, and an online softmax folds them into a 64 x 512 float accumulator in
// registers.  Rows whose index or page is out of range are zero and take no
// weight.  Splits of a query are combined by the log-sum-exp merge.
#include <math.h>

#include "dsa_kernels.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 64;
constexpr int kTile = 16;                        // rows per tile
constexpr int kLatent = kLatentCols;
constexpr int kSsStride = kTile + 1;

template <int W>
struct Smem {
    static constexpr int kQStride = W + 4;
    static constexpr int kRStride = W + 4;
    static constexpr size_t kQ = (size_t)kHeads * kQStride * sizeof(float);
    static constexpr size_t kR = (size_t)kTile * kRStride * sizeof(float);
    static constexpr size_t kS = (size_t)kHeads * kSsStride * sizeof(float);
    static constexpr size_t kStats = 3 * kHeads * sizeof(float);
    static constexpr size_t kRows = kTile * (2 * sizeof(int64_t));
    static constexpr size_t kTotal = kQ + kR + kS + kStats + kRows;
};

__device__ __forceinline__ void widen4(const float* p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
template <int FMT, int W>
__global__ void __launch_bounds__(kThreads)
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
    float* Ss = reinterpret_cast<float*>(smem + S::kRows + S::kQ + S::kR);
    float* m_s = reinterpret_cast<float*>(smem + S::kRows + S::kQ + S::kR + S::kS);
    float* l_s = m_s + kHeads;
    float* alpha_s = l_s + kHeads;

    const int tid = threadIdx.x;
    const int64_t q = blockIdx.y;
    const int split = blockIdx.x;
    QueryInfo qi;
    if (!query_info(b, q, qi, err, /*where=*/33)) {
        if (n_split > 1 && tid < kHeads) {             // no weight in the merge
            part_ml[((q * n_split + split) * kHeads + tid) * 2 + 0] = -INFINITY;
            part_ml[((q * n_split + split) * kHeads + tid) * 2 + 1] = 0.f;
        }
        return;
    }
    int64_t ns = idx == nullptr ? qi.L : n_sel[q];
    if (idx != nullptr) ns = ns < 0 ? 0 : (ns > idx_width ? idx_width : ns);
    const int64_t j_begin = (int64_t)split * rows_per_split;
    const int64_t j_end = j_begin + rows_per_split < ns ? j_begin + rows_per_split : ns;

    constexpr int kQVec = 4;
    const float* qsrc = q_abs + q * (int64_t)kHeads * W;
    for (int v = tid; v < kHeads * (W / kQVec); v += kThreads) {
        const int h = v / (W / kQVec), c = (v % (W / kQVec)) * kQVec;
        *reinterpret_cast<uint4*>(Qs + h * S::kQStride + c) =
            __ldg(reinterpret_cast<const uint4*>(qsrc + (int64_t)h * W + c));
    }
    if (tid < kHeads) { m_s[tid] = -INFINITY; l_s[tid] = 0.f; }

    const int oh = tid >> 2, ocg = tid & 3;            // accumulator owner: head, column group
    float o[kLatent / 4];
#pragma unroll
    for (int i = 0; i < kLatent / 4; ++i) o[i] = 0.f;

    for (int64_t j0 = j_begin; j0 < j_end; j0 += kTile) {
        const int nrows = (int)(j_end - j0 < kTile ? j_end - j0 : kTile);
        if (tid < kTile) {
            int64_t at = -1;
            float2 f = make_float2(0.f, 0.f);
            if (tid < nrows) {
                const int32_t r = idx == nullptr ? (int32_t)(j0 + tid) : idx[q * idx_width + j0 + tid];
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
            const int j = v / kRowVecs, c = (v % kRowVecs) * 16;
            const int64_t at = row_at[j];
            uint4 w = make_uint4(0, 0, 0, 0);
            if (at >= 0) w = __ldg(reinterpret_cast<const uint4*>(pc.codes + at * W + c));
            const float f = at < 0 ? 0.f : (c < kLatent ? row_scale[j].x : row_scale[j].y);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float x[4];
                widen_codes<FMT>(u[k], x);
                *reinterpret_cast<float4*>(Rs + j * S::kRStride + c + 4 * k) =
                    make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
            }
        }
        __syncthreads();
        {                                              // logits: row j, heads h0 + 16 i
            const int j = tid & (kTile - 1), h0 = tid >> 4;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            for (int c = 0; c < W; c += 4) {
                float rf[4];
                widen4(Rs + j * S::kRStride + c, rf);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float qf[4];
                    widen4(Qs + (h0 + 16 * i) * S::kQStride + c, qf);
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[i] = fmaf(qf[k], rf[k], acc[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                Ss[(h0 + 16 * i) * kSsStride + j] = row_at[j] >= 0 ? acc[i] * scale : -INFINITY;
        }
        __syncthreads();
        if (tid < kHeads) {                            // online softmax, one thread per head
            float* srow = Ss + tid * kSsStride;
            const float m_old = m_s[tid];
            float mx = -INFINITY;
            for (int j = 0; j < kTile; ++j) mx = fmaxf(mx, srow[j]);
            const float m_new = fmaxf(m_old, mx);
            float alpha = 1.f, psum = 0.f;
            for (int j = 0; j < kTile; ++j) {
                // no finite maximum yet: rows without weight, or a NaN logit to pass on
                const float p = srow[j] == -INFINITY ? 0.f : expf(srow[j] - m_new);
                srow[j] = p;
                psum += p;
            }
            if (m_new != -INFINITY) alpha = expf(m_old - m_new);
            l_s[tid] = l_s[tid] * alpha + psum;
            m_s[tid] = m_new;
            alpha_s[tid] = alpha;
        }
        __syncthreads();
        {                                              // rescale and accumulate P . R_latent
            const float a = alpha_s[oh];
#pragma unroll
            for (int i = 0; i < kLatent / 4; ++i) o[i] *= a;
            for (int j = 0; j < nrows; ++j) {
                const float p = Ss[oh * kSsStride + j];
                const float* rrow = Rs + j * S::kRStride + 4 * ocg;
#pragma unroll
                for (int i = 0; i < kLatent / 16; ++i) {
                    const float4 r4 = *reinterpret_cast<const float4*>(rrow + 16 * i);
                    o[4 * i + 0] = fmaf(p, r4.x, o[4 * i + 0]);
                    o[4 * i + 1] = fmaf(p, r4.y, o[4 * i + 1]);
                    o[4 * i + 2] = fmaf(p, r4.z, o[4 * i + 2]);
                    o[4 * i + 3] = fmaf(p, r4.w, o[4 * i + 3]);
                }
            }
        }
        __syncthreads();
    }
    __syncthreads();

    const float m = m_s[oh], l = l_s[oh];
    const bool last = n_split == 1;
    const float inv = last ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
    const int64_t part = q * n_split + split;
    float* dst = (last ? out + (q * kHeads + oh) * (int64_t)kLatent
                       : part_o + (part * kHeads + oh) * (int64_t)kLatent) + 4 * ocg;
#pragma unroll
    for (int i = 0; i < kLatent / 16; ++i)
        *reinterpret_cast<float4*>(dst + 16 * i) =
            make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
    if (ocg == 0) {
        if (last) {
            if (lse != nullptr) lse[q * kHeads + oh] = l == 0.f ? -INFINITY : m + logf(l);
        } else {
            part_ml[(part * kHeads + oh) * 2 + 0] = m;
            part_ml[(part * kHeads + oh) * 2 + 1] = l;
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

// CUDA-core splits: enough CTAs to fill the GPU about twice, at least one tile each.
void plan_splits_simt(int32_t n_q, int64_t max_rows, int32_t* rows_per_split, int32_t* n_split) {
    const int64_t target = 2 * (int64_t)sm_count();
    const int64_t tiles = (max_rows + kTile - 1) / kTile;
    int64_t splits = (target + n_q - 1) / n_q;
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
    e = launch_plain(kern, dim3((unsigned)n_split, (unsigned)b.n_q), dim3(kThreads), S::kTotal, st,
                     b, pc, sh.scale, static_cast<const float*>(q_abs), idx, n_sel,
                     sh.index_row_width(), rps, n_split, out, lse, part_o, part_ml, err);
    if (e != cudaSuccess || n_split == 1) return e;
    return launch_merge_splits(b.n_q, n_split, part_o, part_ml, out, lse, st);
}

}  // namespace

void plan_paged_splits(const Shape& sh, const BatchDev& b, int32_t* rows_per_split,
                       int32_t* n_split) {
    int64_t main_rows, max_rows;
    paged_rows(sh, b, &main_rows, &max_rows);
    const int32_t n_q = b.n_q > 0 ? b.n_q : 1;
    if (sh.dtype == DSA_BF16) plan_attention_splits_tc(n_q, main_rows, max_rows, rows_per_split, n_split);
    else plan_splits_simt(n_q, max_rows, rows_per_split, n_split);
}

size_t paged_mla_scratch_bytes(const Shape& sh, const BatchDev& b) {
    int32_t rps, n_split;
    plan_paged_splits(sh, b, &rps, &n_split);
    if (n_split == 1) return 0;
    return (size_t)b.n_q * n_split * kHeads * (kLatent + 2) * sizeof(float);
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
