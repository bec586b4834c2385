// paged_mla_tc.cu -- absorbed-MLA attention over the paged 8-bit cache on the
// tcgen05 tensor cores (bf16 queries).
//
// z[h,j] = scale * q[h,:] . row_j, p = softmax_j(z), out[h,c] = sum_j p[h,j]
// row_j[c] for the 512 latent columns, a row being its 8-bit codes times its
// page's power-of-two scales: both factors are exact in bf16, so the rows are
// widened to bf16 without rounding and only q . row and P . row are formed in
// float32 from exact products.
//
// One CTA takes a range of one query's rows in tiles of 64, two bf16 row
// buffers deep:
//   warps 4-11  load the tile's rows through the block table (four threads a
//               row, each 16 codes of every 64-column block, a tile ahead in
//               registers), widen them and store them in the 128-byte swizzle.
//               A buffer is handed over in pieces of 128 columns: a piece is
//               refilled as soon as the value product has read it, and the next
//               scores start as soon as their first piece is in;
//   warp 12     issues S^T = R . Q^T (M = 64 rows, N = 64 heads, K = the row)
//               and O^T += R^T . P^T (M = 128 latent columns, K = 64 rows), the
//               scores of tile t + 1 before the values of tile t;
//   warps 0-3   softmax: a 16x64b load gives every lane a row and the 32 heads
//               of one parity; running maxima raised only past a slack of 2^8
//               (and O^T rescaled in TMEM then), P as bf16 hi + lo, 2^-18 of it.
// An M = 128 MMA of N = 64 takes 51 cycles and one of N = 128 takes 67 (measured
// back to back on one SM): the cost is reading the row operand.  So where TMEM
// has room (two of the four latent blocks: 2 x 64 columns of scores, 2 x 128 and
// 2 x 64 of output) hi and lo are one product of N = 128 whose halves are added
// in the epilogue, and two products of N = 64 elsewhere.
// Splits of one query are combined by the log-sum-exp merge: a launch over the
// partials, or, for two splits, the two CTAs of a cluster through distributed
// shared memory.
#include <math.h>

#include <cooperative_groups.h>

#include "dsa_kernels.cuh"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace dsa {
namespace {

using namespace sm100;

constexpr int kHeads = 64;
constexpr int kTileRows = 64;
constexpr int kLatent = kLatentCols;
constexpr int kLatentBlocks = 4;                     // of 128 columns (MMA M)
constexpr int kWideBlocks = 2;                       // of them with P hi and lo in one product
constexpr uint32_t kBlock = 64 * 128;                // 64 rows or heads x 64 bf16 columns: 8 KB
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0;                        // S^T of buffer b: 64 b
constexpr uint32_t kOCol = 128;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;                        // lazy rescale threshold (log2 units)
constexpr float kNoMax = -3.0e38f;                   // running maximum before any row
constexpr int kSoftmaxThreads = 128;
constexpr int kLoaders = 256;
constexpr int kThreads = kSoftmaxThreads + kLoaders + 32;
constexpr int kMmaWarp = (kSoftmaxThreads + kLoaders) / 32;

// First TMEM column of latent block i: hi at +0 (and lo at +64 in a wide one).
__host__ __device__ constexpr uint32_t o_col(int i) {
    return kOCol + 64u * (uint32_t)(i < kWideBlocks ? 2 * i : kWideBlocks + i);
}
static_assert(o_col(kLatentBlocks - 1) + 64 == kTmemCols, "TMEM budget");

template <int W>
struct Cfg {
    static constexpr int kCB = W / 64;               // 64-column blocks of a row
    static constexpr int kPieces = (kCB + 1) / 2;    // handed over 128 columns at a time
    static constexpr uint32_t kOffQ = 0;
    static constexpr uint32_t kOffR = kCB * kBlock;
    static constexpr uint32_t kBufBytes = kCB * kBlock;
    // P_hi^T [64 rows x 64 heads] of buffer b: the buffer's rope block, which the
    // scores no longer need, or its own.  P_lo^T: one block, written once the
    // previous tile's value products are done.  It lies behind both P_hi.
    static constexpr uint32_t kOffPx = kOffR + 2 * kBufBytes;
    static constexpr uint32_t kOffPlo = W == 576 ? kOffPx : kOffPx + 2 * kBlock;
    static constexpr uint32_t kOffBar = kOffPlo + kBlock;       // up to 32 barriers
    static constexpr uint32_t kOffValid = kOffBar + 256;        // [2][64] bytes
    static constexpr uint32_t kOffRed = kOffValid + 128;        // [4][64] int
    static constexpr uint32_t kOffL = kOffRed + 4 * 64 * 4;     // [64] float
    static constexpr uint32_t kOffM = kOffL + 64 * 4;           // [64] float
    static constexpr uint32_t kOffMisc = kOffM + 64 * 4;
    static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory budget");
    __host__ __device__ static constexpr uint32_t off_p(int b) {
        return W == 576 ? kOffR + b * kBufBytes + 8 * kBlock : kOffPx + b * kBlock;
    }
};

__device__ __forceinline__ int fkey(float f) {           // order-preserving float -> int
    const int i = __float_as_int(f);
    return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float fval(int k) { return __int_as_float(k >= 0 ? k : k ^ 0x7fffffff); }

// Sixteen codes times their scale as bf16 (exact), two 16-byte pieces.
template <int FMT>
__device__ __forceinline__ void widen16(const uint4& w, float f, uint4 (&r)[2]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[4];
        widen_codes<FMT>(u[i], x);
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0] * f, x[1] * f);
        const __nv_bfloat162 c = __floats2bfloat162_rn(x[2] * f, x[3] * f);
        o[2 * i] = *reinterpret_cast<const uint32_t*>(&a);
        o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&c);
    }
    r[0] = make_uint4(o[0], o[1], o[2], o[3]);
    r[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// True in every softmax thread if `v` is true in any (named barrier 1).
__device__ __forceinline__ bool softmax_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)v), "n"(kSoftmaxThreads) : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
}

// Maxima of x[0..31] over the 16 lanes of a parity by a halving exchange: at
// each step a lane keeps half of its values, swaps the other half with its
// partner across one lane bit and takes the maximum (30 shuffles in all); it
// ends with those of x[e0] and x[e0 + 1], e0 = 2 (lane & 1) + 4 ((lane >> 2) & 7).
__device__ __forceinline__ float2 halving_max(const float (&x)[32], int lane) {
    float a[16], b[8], c[4], d[2];
    const bool h4 = (lane >> 4) & 1, h3 = (lane >> 3) & 1, h2 = (lane >> 2) & 1, h0 = lane & 1;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        a[i] = fmaxf(h4 ? x[i + 16] : x[i], __shfl_xor_sync(0xffffffffu, h4 ? x[i] : x[i + 16], 16));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        b[i] = fmaxf(h3 ? a[i + 8] : a[i], __shfl_xor_sync(0xffffffffu, h3 ? a[i] : a[i + 8], 8));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = fmaxf(h2 ? b[i + 4] : b[i], __shfl_xor_sync(0xffffffffu, h2 ? b[i] : b[i + 4], 4));
#pragma unroll
    for (int i = 0; i < 2; ++i)
        d[i] = fmaxf(h0 ? c[i + 2] : c[i], __shfl_xor_sync(0xffffffffu, h0 ? c[i] : c[i + 2], 1));
    return make_float2(d[0], d[1]);
}

template <int FMT, int W>
__global__ void __launch_bounds__(kThreads, 1)
paged_mla_tc(const __grid_constant__ CUtensorMap tm_q, PagedCache pc, BatchDev b, float scale,
             const int32_t* __restrict__ idx, const int32_t* __restrict__ n_sel, int64_t idx_width,
             int32_t rows_per_split, int32_t n_split, int32_t pair, float* __restrict__ out,
             float* __restrict__ lse, float* __restrict__ part_o, float* __restrict__ part_ml,
             int32_t* err) {
    using C = Cfg<W>;
    constexpr int kParts = W > kLatent ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t *q_full = bars, *drain = bars + 1, *s_full = bars + 2, *p_full = bars + 4,
             *r_full = bars + 6,                     // [buffer][piece]
             *freed = bars + 16;                     // [buffer][latent block]: its values are in
    uint8_t* valid = smem + C::kOffValid;
    int* red = reinterpret_cast<int*>(smem + C::kOffRed);
    float* l_fin = reinterpret_cast<float*>(smem + C::kOffL);
    float* m_fin = reinterpret_cast<float*>(smem + C::kOffM);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t q = blockIdx.y;
    const int split = blockIdx.x;
    // Two CTAs per split (gridDim.z == 2) both form the scores and divide the
    // value product and the output by latent half.
    const int half = blockIdx.z;
    const bool halved = gridDim.z == 2;
    auto owns = [&](int blk) { return !halved || (blk >> 1) == half; };
    // Two splits of a query as a cluster: each stages its unnormalised O as
    // [head][latent] in its shared memory, then combines half of the heads from
    // both through distributed shared memory and writes the final output.
    // Every thread of both CTAs calls this once (an empty split with l = 0).
    float* stage = reinterpret_cast<float*>(smem);
    auto pair_merge = [&]() {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();                                    // both stages are written
        const int rank = (int)cl.block_rank();
        const float4* st0 = reinterpret_cast<const float4*>(stage);
        const float4* st1 = reinterpret_cast<const float4*>(cl.map_shared_rank(stage, rank ^ 1));
        const float* m1p = cl.map_shared_rank(m_fin, rank ^ 1);
        const float* l1p = cl.map_shared_rank(l_fin, rank ^ 1);
        float4* o4 = reinterpret_cast<float4*>(out);
        constexpr int kC4 = kLatent / 4;
        for (int i = threadIdx.x; i < (kHeads / 2) * kC4; i += blockDim.x) {
            const int h = (kHeads / 2) * rank + i / kC4, c4 = i % kC4;
            const float l0 = l_fin[h], l1 = l1p[h];
            const float M = fmaxf(m_fin[h], m1p[h]);  // kNoMax where there was no row
            const float f0 = l0 != 0.f ? exp2f(m_fin[h] - M) : 0.f;
            const float f1 = l1 != 0.f ? exp2f(m1p[h] - M) : 0.f;
            const float L = l0 * f0 + l1 * f1;
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            if (L != 0.f) {
                const float inv = 1.f / L;
                const float4 a = l0 != 0.f ? st0[h * kC4 + c4] : r;
                const float4 c = l1 != 0.f ? st1[h * kC4 + c4] : r;
                r = make_float4((a.x * f0 + c.x * f1) * inv, (a.y * f0 + c.y * f1) * inv,
                                (a.z * f0 + c.z * f1) * inv, (a.w * f0 + c.w * f1) * inv);
            }
            o4[(q * kHeads + h) * kC4 + c4] = r;
            if (c4 == 0 && lse != nullptr)
                lse[q * kHeads + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        }
        cl.sync();                                    // the peer's reads of this stage are done
    };

    if (threadIdx.x < kHeads) { m_fin[threadIdx.x] = kNoMax; l_fin[threadIdx.x] = 0.f; }
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(drain, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kSoftmaxThreads);
            for (int g = 0; g < C::kPieces; ++g) mbar_init(&r_full[i * C::kPieces + g], kLoaders);
            for (int g = 0; g < kLatentBlocks; ++g) mbar_init(&freed[i * kLatentBlocks + g], 1);
        }
        fence_mbarrier_init();
    }
    if (warp == kMmaWarp) {
        if (lane == 0) prefetch_tensormap(&tm_q);
        __syncwarp();
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    auto leave = [&]() {
        tc_fence_before();
        __syncthreads();
        if (warp == kMmaWarp) {
            tc_fence_after();
            tmem_dealloc(tmem_base, kTmemCols);
        }
    };
    pdl_wait();                                       // everything read below may be an earlier kernel's
    pdl_trigger();

    // Row j of the query's list.  The loaders read the entries of their first
    // three tiles before the list's length is known (none past its width).
    const bool dense = idx == nullptr;
    const int64_t j0 = (int64_t)split * rows_per_split;
    const int row = (threadIdx.x - kSoftmaxThreads) >> 2, k4 = threadIdx.x & 3;
    const bool loader = warp >= kSoftmaxThreads / 32 && warp < kMmaWarp;
    auto entry = [&](int t, int64_t end) -> int32_t {
        const int64_t j = j0 + (int64_t)t * kTileRows + row;
        return j >= end ? -1 : (dense ? (int32_t)j : idx[q * idx_width + j]);
    };
    int32_t e0 = -1, e1 = -1, e2 = -1;                // entries of tiles t, t + 1, t + 2
    if (loader) {
        const int64_t end = dense ? INT64_MAX : idx_width;
        e0 = entry(0, end);
        e1 = entry(1, end);
        e2 = entry(2, end);
    }
    int64_t ns = dense ? 0 : n_sel[q];
    QueryInfo qi;
    const bool known = query_info(b, q, qi, err, /*where=*/34);
    if (dense) ns = known ? qi.L : 0;
    else ns = ns < 0 ? 0 : (ns > idx_width ? idx_width : ns);
    const int64_t j1 = j0 + rows_per_split < ns ? j0 + rows_per_split : ns;
    if (!known || j0 >= j1) {
        if (pair) {                                   // no weight from this half
            __syncthreads();
            if (known) pair_merge();
        } else if (n_split == 1) {                    // no rows: out = 0, lse = -inf
            if (known) {
                for (int i = threadIdx.x; i < kHeads * kLatent; i += blockDim.x)
                    out[q * kHeads * kLatent + i] = 0.f;
                if (lse != nullptr && threadIdx.x < kHeads) lse[q * kHeads + threadIdx.x] = -INFINITY;
            }
        } else if (threadIdx.x < kHeads && half == 0) {  // no weight in the merge
            const int64_t part = q * n_split + split;
            part_ml[(part * kHeads + threadIdx.x) * 2] = -INFINITY;
            part_ml[(part * kHeads + threadIdx.x) * 2 + 1] = 0.f;
        }
        leave();
        return;
    }
    const int n_tiles = (int)((j1 - j0 + kTileRows - 1) / kTileRows);

    if (loader) {                                                     // ---- loads
        // A row's way to its codes is three dependent reads (list entry, block
        // table, codes and scales): the entries are read three tiles ahead, the
        // table two, the codes one.
        const int32_t* table = pc.block_table + (int64_t)qi.seq * pc.pg.table_ld;
        auto page_at = [&](int t, int32_t r) -> int32_t {
            const int64_t j = j0 + (int64_t)t * kTileRows + row;
            if (j >= j1) return -1;
            int32_t p = -1;
            if (r >= 0 && r < qi.L && (r >> pc.pg.shift) < pc.pg.table_ld) p = table[r >> pc.pg.shift];
            return p;
        };
        struct Place { const uint8_t* codes; float f0, f1; };
        // the row's codes and scales; reports a row of the list that has no page
        auto place = [&](int t, int32_t r, int32_t page) -> Place {
            Place p{nullptr, 0.f, 0.f};
            if (page >= 0 && page < pc.pg.n_pages) {
                const int64_t at = ((int64_t)page << pc.pg.shift) + (r & (pc.pg.page_rows - 1));
                p.codes = pc.codes + at * W + 16 * k4;
                p.f0 = e8m0(pc.scales[(int64_t)page * kParts]);
                if (kParts == 2) p.f1 = e8m0(pc.scales[(int64_t)page * kParts + 1]);
            } else if (j0 + (int64_t)t * kTileRows + row < j1) {
                record_error(err, kDevBadIndex, (int32_t)q, /*where=*/34);
            }
            return p;
        };
        auto fetch = [&](const Place& p, int cb) -> uint4 {
            return p.codes != nullptr ? __ldg(reinterpret_cast<const uint4*>(p.codes + 64 * cb))
                                      : make_uint4(0, 0, 0, 0);
        };
        if (j0 + row >= j1) e0 = -1;
        if (j0 + kTileRows + row >= j1) e1 = -1;
        if (j0 + 2 * kTileRows + row >= j1) e2 = -1;
        int32_t p0 = page_at(0, e0), p1 = page_at(1, e1);
        Place cur = place(0, e0, p0);
        uint4 raw[C::kCB];
#pragma unroll
        for (int cb = 0; cb < C::kCB; ++cb) raw[cb] = fetch(cur, cb);
        int32_t p2 = page_at(2, e2), e3 = n_tiles > 3 ? entry(3, j1) : -1;
        bool ok = true;
        for (int t = 0; t < n_tiles && ok; ++t) {
            const int buf = t & 1;
            const Place nxt = t + 1 < n_tiles ? place(t + 1, e1, p1) : Place{nullptr, 0.f, 0.f};
            uint8_t* rbuf = smem + C::kOffR + buf * C::kBufBytes + row * 128;
#pragma unroll
            for (int g = 0; g < C::kPieces; ++g) {
                // the piece's columns have been read by tile t - 2's value
                // product (the rope block, which held its P_hi, by all of it)
                if (t >= 2 && ok)
                    ok = mbar_wait(&freed[buf * kLatentBlocks + (g < kLatentBlocks ? g : kLatentBlocks - 1)],
                                   (uint32_t)(((t >> 1) - 1) & 1), kWaitNs);
                if (!ok) break;
                if (g == 0 && k4 == 0) valid[buf * kTileRows + row] = cur.codes != nullptr;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int cb = 2 * g + c;
                    if (cb >= C::kCB) continue;
                    uint4 x[2];
                    widen16<FMT>(raw[cb], cb < kLatent / 64 ? cur.f0 : cur.f1, x);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<uint4*>(rbuf + cb * kBlock + (((2 * k4 + k) ^ (row & 7)) << 4)) =
                            x[k];
                    raw[cb] = fetch(nxt, cb);
                }
                fence_proxy_async_smem();
                mbar_arrive(&r_full[buf * C::kPieces + g]);
            }
            cur = nxt;
            e1 = e2; p1 = p2;
            e2 = e3;
            p2 = t + 3 < n_tiles ? page_at(t + 3, e2) : -1;
            e3 = t + 4 < n_tiles ? entry(t + 4, j1) : -1;
        }
        if (!ok && threadIdx.x == kSoftmaxThreads) record_error(err, kDevTimeout, (int32_t)q, /*where=*/35);
    } else if (warp == kMmaWarp) {                                    // ---- query load, MMA issue
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, C::kCB * kBlock);
            for (int cb = 0; cb < C::kCB; ++cb)
                tma_load_2d(smem + C::kOffQ + cb * kBlock, &tm_q, q_full, 64 * cb, (int32_t)(q * kHeads));
            constexpr uint32_t idesc_s = idesc_bf16_f32(kTileRows, kHeads);
            constexpr uint32_t idesc_pv = idesc_bf16_f32_major(128, kHeads, 1, 1);
            constexpr uint32_t idesc_pv2 = idesc_bf16_f32_major(128, 2 * kHeads, 1, 1);
            const uint32_t base = smem_u32(smem);
            const uint64_t d_q = sdesc_kmajor_sw128(base + C::kOffQ);
            bool ok = mbar_wait(q_full, 0, kWaitNs);
            int next_s = 0, next_v = 0;
            uint64_t t_prog = globaltimer_ns();
            while (ok && next_v < n_tiles) {
                bool progressed = false;
                if (next_s < n_tiles && next_s <= next_v + 1 &&
                    mbar_test_wait(&r_full[(next_s & 1) * C::kPieces], (uint32_t)((next_s >> 1) & 1))) {
                    // S^T(s) = R(s) Q^T, piece by piece as they come in
                    const int bs = next_s & 1;
                    const uint64_t d_r = sdesc_kmajor_sw128(base + C::kOffR + bs * C::kBufBytes);
#pragma unroll
                    for (int g = 0; g < C::kPieces; ++g) {
                        if (g > 0 && ok)
                            ok = mbar_wait(&r_full[bs * C::kPieces + g], (uint32_t)((next_s >> 1) & 1), kWaitNs);
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int cb = 2 * g + k / 4, kk = k & 3;
                            if (cb >= C::kCB) continue;
                            const uint64_t o = (cb * kBlock + kk * 32) >> 4;
                            mma_bf16_ss(tmem_base + kSCol + 64 * bs, d_r + o, d_q + o, idesc_s,
                                        (cb | kk) != 0 ? 1u : 0u);
                        }
                    }
                    mma_commit(&s_full[bs]);
                    ++next_s;
                    progressed = true;
                }
                if (next_v < next_s &&
                    mbar_test_wait(&p_full[next_v & 1], (uint32_t)((next_v >> 1) & 1))) {
                    // A = R^T: MN-major, 64-column blocks 8 KB apart, 8-row
                    // groups 1 KB apart.  B = P^T: MN-major, 64 heads a block,
                    // lo's block behind hi's.
                    tc_fence_after();
                    const int bv = next_v & 1;
                    const uint32_t p_hi = base + C::off_p(bv), p_lo = base + C::kOffPlo;
                    const uint64_t d_a = sdesc_sw128(base + C::kOffR + bv * C::kBufBytes, kBlock, 1024);
                    const uint64_t d_both = sdesc_sw128(p_hi, p_lo - p_hi, 1024);
                    const uint64_t d_hi = sdesc_sw128(p_hi, 1024, 1024), d_lo = sdesc_sw128(p_lo, 1024, 1024);
                    const uint32_t acc = next_v > 0 ? 1u : 0u;
#pragma unroll
                    for (int i = 0; i < kLatentBlocks; ++i) {
                        if (owns(i)) {
#pragma unroll
                            for (int kk = 0; kk < kTileRows / 16; ++kk) {
                                const uint64_t oa = (2 * i * kBlock + kk * 2048) >> 4, ob = (kk * 2048) >> 4;
                                if (i < kWideBlocks) {
                                    mma_bf16_ss(tmem_base + o_col(i), d_a + oa, d_both + ob, idesc_pv2,
                                                kk > 0 ? 1u : acc);
                                } else {
                                    mma_bf16_ss(tmem_base + o_col(i), d_a + oa, d_hi + ob, idesc_pv,
                                                kk > 0 ? 1u : acc);
                                    mma_bf16_ss(tmem_base + o_col(i), d_a + oa, d_lo + ob, idesc_pv, 1u);
                                }
                            }
                        }
                        mma_commit(&freed[bv * kLatentBlocks + i]);
                    }
                    ++next_v;
                    progressed = true;
                }
                if (progressed) t_prog = globaltimer_ns();
                else if (globaltimer_ns() - t_prog > kWaitNs) ok = false;
            }
            if (!ok) record_error(err, kDevTimeout, (int32_t)q, /*where=*/36);
            mma_commit(drain);
            mbar_wait(drain, 0, 50000000ull);
        }
    } else {                                                          // ---- softmax
        // The scores of an M = 64 tile sit in lanes 0..15 of TMEM quadrant wq;
        // lane l of warp wq takes row 16 wq + (l >> 2) + 8 (l & 1) and the heads
        // of parity p = (l >> 1) & 1.
        const int wq = warp;
        const int p = (lane >> 1) & 1;
        const int srow = 16 * wq + (lane >> 2) + 8 * (lane & 1);
        const uint32_t lane_addr = tmem_base + ((uint32_t)(32 * wq) << 16);
        const float c2 = scale * kLog2e;
        float l_part[32];                            // row sums of heads 32 p .. 32 p + 31
#pragma unroll
        for (int e = 0; e < 32; ++e) l_part[e] = 0.f;
        float* m_sh = m_fin;                         // running maxima, one writer per head
        float* alpha_s = l_fin;                      // rescale factors
        bool ok = true;
        for (int t = 0; t < n_tiles; ++t) {
            const int bf = t & 1;
            if (ok) ok = mbar_wait(&s_full[bf], (uint32_t)((t >> 1) & 1), kWaitNs);
            tc_fence_after();
            const bool has_row = valid[bf * kTileRows + srow] != 0;
            float x[32];                             // x[k]: head p + 2 k
            {
                float v[32];
                tmem_ld_16x64b_32(lane_addr + kSCol + 64 * bf, v);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = has_row ? v[e] * c2 : -INFINITY;
            }
            bool exceed = false;
#pragma unroll
            for (int e = 0; e < 32; ++e) exceed |= x[e] > m_sh[p + 2 * e] + kSlack;
            bool any_raised = false;
            if (softmax_any(exceed)) {
                const float2 mx = halving_max(x, lane);
                const int e0 = 2 * (lane & 1) + 4 * ((lane >> 2) & 7);
                int* rb = red + wq * kHeads;
                rb[p + 2 * e0] = fkey(mx.x);
                rb[p + 2 * e0 + 2] = fkey(mx.y);
                softmax_sync();
                bool raised = false;
                if (threadIdx.x < kHeads) {            // raise this head's running maximum?
                    const int h = threadIdx.x;
                    const float tmax = fval(max(max(red[h], red[kHeads + h]),
                                                max(red[2 * kHeads + h], red[3 * kHeads + h])));
                    const float m_old = m_sh[h];
                    float a = 1.f;
                    if (tmax > m_old + kSlack) {
                        a = exp2f(m_old - tmax);       // 0 from kNoMax
                        m_sh[h] = tmax;
                        raised = true;
                    }
                    alpha_s[h] = a;
                }
                any_raised = softmax_any(raised);
            }
            if (any_raised) {
#pragma unroll
                for (int e = 0; e < 32; ++e) l_part[e] *= alpha_s[32 * p + e];
                if (t > 0) {                           // O^T follows the new maxima
                    const int pb = (t - 1) & 1;
                    if (ok) ok = mbar_wait(&freed[pb * kLatentBlocks + kLatentBlocks - 1],
                                           (uint32_t)(((t - 1) >> 1) & 1), kWaitNs);
                    tc_fence_after();
                    // 32 columns at a time: four of each wide block, two of the others
#pragma unroll 1
                    for (int k = 0; k < 2 * (kLatentBlocks + kWideBlocks); ++k) {
                        const int blk = k < 4 * kWideBlocks ? k >> 2 : kWideBlocks + ((k - 4 * kWideBlocks) >> 1);
                        if (!owns(blk)) continue;
                        const uint32_t a = lane_addr + kOCol + 32 * k;
                        const int hh = 32 * (k & 1);
                        float v[32];
                        tmem_ld_32cols(a, v);
#pragma unroll
                        for (int c = 0; c < 32; ++c) v[c] *= alpha_s[hh + c];
                        tmem_st_32cols(a, v);
                    }
                    tc_fence_before();
                }
                softmax_sync();                        // alpha_s is read, O^T rescaled
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = exp2f(x[e] - m_sh[p + 2 * e]);
            // P^T row: this lane and lane ^ 2 (same row, other parity) swap
            // halves, so that this lane holds heads 32 p .. 32 p + 31 in pairs;
            // p = hi + lo with hi = bf16(p), lo = bf16(p - hi).
            uint8_t* prow = smem + C::off_p(bf) + srow * 128;
            uint8_t* plow = smem + C::kOffPlo + srow * 128;
            uint32_t lo4[4][4];
#pragma unroll
            for (int c16 = 0; c16 < 4; ++c16) {
                uint32_t w4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int k = 4 * c16 + e;
                    const float r = __shfl_xor_sync(0xffffffffu, p ? x[k] : x[k + 16], 2);
                    const float a = p ? r : x[k], c = p ? x[k + 16] : r;
                    const __nv_bfloat162 hi = __floats2bfloat162_rn(a, c);
                    const float2 hf = __bfloat1622float2(hi);
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(a - hf.x, c - hf.y);
                    const float2 lf = __bfloat1622float2(lo);
                    l_part[2 * k] += hf.x + lf.x;      // the weights the products use
                    l_part[2 * k + 1] += hf.y + lf.y;
                    w4[e] = *reinterpret_cast<const uint32_t*>(&hi);
                    lo4[c16][e] = *reinterpret_cast<const uint32_t*>(&lo);
                }
                *reinterpret_cast<uint4*>(prow + (((4 * p + c16) ^ (srow & 7)) << 4)) =
                    make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
            // the previous tile's value products read P_lo
            if (t > 0 && ok)
                ok = mbar_wait(&freed[((t - 1) & 1) * kLatentBlocks + kLatentBlocks - 1],
                               (uint32_t)(((t - 1) >> 1) & 1), kWaitNs);
#pragma unroll
            for (int c16 = 0; c16 < 4; ++c16)
                *reinterpret_cast<uint4*>(plow + (((4 * p + c16) ^ (srow & 7)) << 4)) =
                    make_uint4(lo4[c16][0], lo4[c16][1], lo4[c16][2], lo4[c16][3]);
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(&p_full[bf]);
        }
        {
            const int tl = n_tiles - 1;
            if (ok) ok = mbar_wait(&freed[(tl & 1) * kLatentBlocks + kLatentBlocks - 1],
                                   (uint32_t)((tl >> 1) & 1), kWaitNs);
        }
        if (!ok) record_error(err, kDevTimeout, (int32_t)q, /*where=*/37);
        // row sums to shared memory (the row buffers are free now)
        float* lsc = reinterpret_cast<float*>(smem + C::kOffR);
#pragma unroll
        for (int e = 0; e < 32; ++e) lsc[srow * (kHeads + 1) + 32 * p + e] = l_part[e];
    }

    // ---- epilogue, warps 0-7: per-head sums, then O^T read out of TMEM
    if (warp < 8) {
        asm volatile("bar.sync 3, 256;" ::: "memory");
        tc_fence_after();
        const int wq = warp & 3, sg = warp >> 2;
        const int hb = 32 * sg;                      // this warp's heads
        const bool head_owner = warp < 2;            // head 32 warp + lane
        const int ho = threadIdx.x;
        const uint32_t lane_addr = tmem_base + ((uint32_t)(32 * wq) << 16);
        const float* lsc = reinterpret_cast<const float*>(smem + C::kOffR);
        if (head_owner) {
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int r = 0; r < kTileRows; ++r) s4[r & 3] += lsc[r * (kHeads + 1) + ho];
            l_fin[ho] = (s4[0] + s4[1]) + (s4[2] + s4[3]);
        }
        asm volatile("bar.sync 3, 256;" ::: "memory");
        const bool final_out = n_split == 1;
        const int64_t part = q * n_split + split;
        float* dst = pair ? stage
                          : (final_out ? out + q * kHeads * kLatent : part_o + part * kHeads * kLatent);
        // lane 32 wq + lane of block i holds latent column 128 i + 32 wq + lane
#pragma unroll
        for (int i = 0; i < kLatentBlocks; ++i) {
            if (!owns(i)) continue;
            const int c = 128 * i + 32 * wq + lane;
            float v[32];
            if (i < kWideBlocks) {                   // hi and lo halves
                float u[32];
                tmem_ld_32cols_x2(lane_addr + o_col(i) + hb, lane_addr + o_col(i) + 64 + hb, v, u);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] += u[e];
            } else {
                tmem_ld_32cols(lane_addr + o_col(i) + hb, v);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float l = l_fin[hb + e];
                const float inv = final_out ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                dst[(hb + e) * kLatent + c] = v[e] * inv;
            }
        }
        if (head_owner && !pair && half == 0) {
            const float l = l_fin[ho], m = m_fin[ho];
            if (final_out) {
                if (lse != nullptr) lse[q * kHeads + ho] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                part_ml[(part * kHeads + ho) * 2] = l == 0.f ? -INFINITY : m * kLn2;
                part_ml[(part * kHeads + ho) * 2 + 1] = l;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (pair) pair_merge();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

template <int FMT, int W>
cudaError_t launch_w(const Shape& sh, const BatchDev& b, const PagedCache& pc, const void* q_abs,
                     const int32_t* idx, const int32_t* n_sel, float* out, float* lse,
                     float* part_o, float* part_ml, int32_t rps, int32_t n_split, int32_t* err,
                     cudaStream_t st) {
    using C = Cfg<W>;
    CUtensorMap tm_q;
    const uint64_t dims[2] = {(uint64_t)W, (uint64_t)b.n_q * kHeads};
    const uint64_t strides[1] = {(uint64_t)W * 2};
    const uint32_t box[2] = {64, kHeads};
    if (!encode_bf16_map(&tm_q, q_abs, 2, dims, strides, box)) return cudaErrorInvalidValue;
    auto kern = paged_mla_tc<FMT, W>;
    cudaError_t e = ensure_dyn_smem((const void*)kern, (int)C::kSmemBytes);
    if (e != cudaSuccess) return e;
    const int32_t pair = n_split == 2 ? 1 : 0;
    // a launch of few CTAs doubles them by latent half while it fits one wave
    const unsigned halves =
        n_split > 2 && (int64_t)b.n_q * n_split * 2 <= (int64_t)sm_count() ? 2u : 1u;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_split, (unsigned)b.n_q, halves);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pair ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, tm_q, pc, b, sh.scale, idx, n_sel, sh.index_row_width(), rps,
                           n_split, pair, out, lse, part_o, part_ml, err);
    if (e != cudaSuccess || n_split <= 2) return e;
    return launch_merge_splits(b.n_q, n_split, part_o, part_ml, out, lse, st);
}

}  // namespace

cudaError_t launch_paged_mla_tc(const Shape& sh, const BatchDev& b, const PagedCache& pc,
                                const void* q_abs, const int32_t* idx, const int32_t* n_sel,
                                float* out, float* lse, float* part_o, float* part_ml, int32_t rps,
                                int32_t n_split, int32_t* err, cudaStream_t st) {
    const bool wide = sh.width() == 576;
    auto f = pc.pg.format == DSA_CACHE_E4M3 ? (wide ? launch_w<DSA_CACHE_E4M3, 576> : launch_w<DSA_CACHE_E4M3, 512>)
                                            : (wide ? launch_w<DSA_CACHE_S8, 576> : launch_w<DSA_CACHE_S8, 512>);
    return f(sh, b, pc, q_abs, idx, n_sel, out, lse, part_o, part_ml, rps, n_split, err, st);
}

}  // namespace dsa
