// paged_mla_tc.cu -- absorbed-MLA attention over the paged 8-bit cache on the
// tcgen05 tensor cores (bf16 queries).
//
// z[h,j] = scale * q[h,:] . row_j, p = softmax_j(z), out[h,c] = sum_j p[h,j]
// row_j[c] for the 512 latent columns, a row being its 8-bit codes times its
// page's power-of-two scales 2^e (latent) and 2^r (rope).  The tensor cores see
// the codes themselves: both formats are exact in f16, so a row is widened with
// one conversion per two codes and its scales are applied to sums in float32,
//     z = scale (2^e S_lat + 2^r S_rope),
//     out = sum_j w_j codes_j / sum_j p_j,  w_j = p_j 2^e_j,
// with w kept relative to a running maximum of z + e (a row's weight in the
// output), and p relative to the same maximum with one fixed exponent taken off
// (kEBase: every exponent a scale may have then keeps p within float32).
// The query becomes f16 times one power of two for all its heads: exact for elements
// down to 2^-31 of the largest, to 2^-39 of it below that.  (A power for each head, where
// their sizes differ much, was measured: the branch on it among a tile's scores cost
// 1,024 queries 695 -> 786 us.)  w is
// carried as two f16 parts, hi + lo, to 2^-22 of it or 2^-37 of the largest.
//
// One CTA takes a range of one query's rows in tiles of 64, two f16 row buffers
// deep:
//   warps 8-15  load the tile's rows through the block table, eight rows a warp,
//               two tiles ahead in registers, widen them and store them in the
//               128-byte swizzle.  A buffer is handed over in pieces of 128
//               columns, all warps on one piece after the other: a piece is
//               refilled as soon as the value product has read it, and the next
//               scores start as soon as their first is in (5% less time for 64
//               queries of 2,048 rows than with two warps to each piece);
//   warp 16     issues S^T = R . Q^T (M = 64 rows, N = 64 heads, K = the row)
//               and O^T += R^T . W^T (M = 128 latent columns, K = 64 rows), the
//               scores of tile t + 1 before the values of tile t;
//   warps 0-7   softmax: a 16x64b load gives every lane a row and 16 heads (the
//               query's rows are laid out so that they are neighbours); maxima
//               are raised only past a slack, and those heads' columns of O^T
//               rescaled in TMEM then.
// Operand reads from shared memory bound the MMAs (128 bytes a cycle; measured
// back to back on one SM: M = 64, N = 64 34 cycles, M = 128 with N = 64 50 and with
// N = 128 66).  So where TMEM has room hi and lo are one product of N = 128 whose
// halves are added in the epilogue -- two of the four latent blocks (three without
// rope) -- and two products of N = 64 elsewhere: 2,540 cycles a tile in all.
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
constexpr uint32_t kBlock = 64 * 128;                // 64 rows or heads x 64 f16 columns: 8 KB
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0, kSRopeCol = 64;        // S^T of the latent and the rope columns
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A head's weights are w = 2^(x - m) with a reference m that is set kRoom below the
// largest logit met and set again (and O^T rescaled) only when one exceeds it by more
// than kSlack, all in log2: w is then at least 2^12 for the largest row and at most
// 55,109, within f16, whose step of 2^-24 the weights share: a weight is off by 2^-37 of
// the largest one at most.  (With m at the largest logit itself, every row 2^25 below
// it had no weight: 2,048 equal rows 17 nats below one row of value zero gave zeros.
// What the room costs in raises: 1,024 queries of 2,048 rows 638 us without, 698 us so,
// 64 queries 65.4 and 71.0 us; with a room of 10, 685 and 70.0 us.)
constexpr float kRoom = 12.f, kSlack = 15.75f;
// x = z + (e - kEBase): the reference m is kRoom or more below the largest x, so the
// row there has p = 2^(x - m - (e - kEBase)) >= 2^-115 (e <= 119), 2^34 of float32's
// smallest steps.  A row of so small a scale that x says little of its p counts
// for m as if its x were z - kLift, which keeps p <= 2^101.75 and sums of 2^25 such
// rows within float32; its w, at 2^16 less than another's for the append's smallest
// exponent, is still good to 2^-21.  x is rounded with the exponent in it, to 2^-24 of
// its size: kEBase is the exponent of pages of values up to 1.75 (e4m3), so that this
// is z's own rounding for usual caches.
constexpr int kEBase = -8;
constexpr float kLift = 86.f;
// w stands in for p (times 2^(kEBase - e)) while neither is lost below 2^-126: rows of
// x - z above kSmall, m set by rows of x - z up to kLarge (p >= 2^-36 there).
constexpr float kSmall = -60.f, kLarge = 48.f;
// Tiles whose values are summed in TMEM before the sum moves to memory (to the
// CTA's own part of the output or of the partials).  The tensor cores cut each
// accumulation off instead of rounding it, so a sum's error grows with the tiles
// in it: relative to the output, against 64 bits, 0.3e-6 for 2 tiles, 1.2e-6 for
// 16, 1.6e-6 for 32, where float32 sums have 0.5e-6.  Moved every 11 tiles it is
// 0.9e-6 for 32, at a cost: 1,024 queries of 2,048 rows take 650 us without and
// 698 us so (every 16 tiles 673 us, and errors above 1e-6).
constexpr int kFlushTiles = 11;
constexpr float kNoMax = -3.0e38f;                   // running maximum before any row
constexpr int kSoftmaxThreads = 256;
constexpr int kLoaders = 256;
constexpr int kThreads = kSoftmaxThreads + kLoaders + 32;
constexpr int kMmaWarp = (kSoftmaxThreads + kLoaders) / 32;
constexpr int kMergers = kSoftmaxThreads + kLoaders;  // threads of the epilogue and the pair merge

template <int W>
struct Cfg {
    static constexpr int kCB = W / 64;               // 64-column blocks of a row
    static constexpr int kPieces = (kCB + 1) / 2;    // handed over 128 columns at a time
    // latent blocks with hi and lo in one product, and O^T's columns: hi at +0
    // (and lo at +64 in a wide block)
    static constexpr int kWide = W == 576 ? 2 : 3;
    static constexpr uint32_t kOCol = W == 576 ? 128 : 64;
    __host__ __device__ static constexpr uint32_t o_col(int i) {
        return kOCol + 64u * (uint32_t)(i < kWide ? 2 * i : kWide + i);
    }
    static_assert(kOCol + 64 * (kWide + kLatentBlocks) == kTmemCols, "TMEM budget");
    static constexpr uint32_t kOffQ = 0;
    static constexpr uint32_t kOffR = kCB * kBlock;
    static constexpr uint32_t kBufBytes = kCB * kBlock;
    // W_hi^T [64 rows x 64 heads] of buffer b: the buffer's rope block, which the
    // scores no longer need, or its own.  W_lo^T: one block, written once the
    // previous tile's value products are done.  It lies behind both W_hi.
    static constexpr uint32_t kOffPx = kOffR + 2 * kBufBytes;
    static constexpr uint32_t kOffPlo = W == 576 ? kOffPx : kOffPx + 2 * kBlock;
    static constexpr uint32_t kOffBar = kOffPlo + kBlock;       // up to 32 barriers
    static constexpr uint32_t kOffRow = kOffBar + 256;          // [2][64] packed scales
    static constexpr uint32_t kOffL = kOffRow + 2 * 64 * 4;     // [64] float
    static constexpr uint32_t kOffM = kOffL + 64 * 4;           // [64] float
    static constexpr uint32_t kOffMs = kOffM + 64 * 4;          // [64] float
    static constexpr uint32_t kOffMf = kOffMs + 64 * 4;         // [64] float
    static constexpr uint32_t kOffMisc = kOffMf + 64 * 4;
    static constexpr uint32_t kSmemBytes = kOffMisc + 64 + 1024;
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

__device__ __forceinline__ float ex2(float x) {          // 2^x, 0 below 2^-126
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 32 bytes of read-only memory (32-byte aligned).
__device__ __forceinline__ void ldg_32bytes(const uint8_t* p, uint32_t (&r)[8]) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7])
                 : "l"(p));
}

// Packed scales of a tile's row: the bytes of its two parts and this flag.
constexpr uint32_t kHasRow = 0x10000u;

// A wait of all lanes of a warp, which go on or give up together: what follows
// synchronises or is .aligned.  (A last test behind the time limit: the whole CTA may
// have been off the multiprocessor meanwhile.  The votes cost 1,024 queries 698 ->
// 708 us.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    const bool in = mbar_wait(bar, parity, kWaitNs) || mbar_try_wait(bar, parity);
    return __all_sync(0xffffffffu, in);
}

__device__ __forceinline__ void softmax_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
}

// Maxima of x[0..15] + lift over the 16 lanes that hold the same heads by a halving
// exchange: at each step a lane keeps half of its values, swaps the other half
// with its partner across one lane bit and takes the maximum; it ends with that
// of x[8 b4 + 4 b3 + 2 b2 + b0], b the bits of its lane.
__device__ __forceinline__ float halving_max(const float (&x)[16], float lift, int lane) {
    float a[8], b[4], c[2];
    const bool h4 = (lane >> 4) & 1, h3 = (lane >> 3) & 1, h2 = (lane >> 2) & 1, h0 = lane & 1;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a[i] = fmaxf((h4 ? x[i + 8] : x[i]) + lift,
                     __shfl_xor_sync(0xffffffffu, (h4 ? x[i] : x[i + 8]) + lift, 16));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        b[i] = fmaxf(h3 ? a[i + 4] : a[i], __shfl_xor_sync(0xffffffffu, h3 ? a[i] : a[i + 4], 8));
#pragma unroll
    for (int i = 0; i < 2; ++i)
        c[i] = fmaxf(h2 ? b[i + 2] : b[i], __shfl_xor_sync(0xffffffffu, h2 ? b[i] : b[i + 2], 4));
    return fmaxf(h0 ? c[1] : c[0], __shfl_xor_sync(0xffffffffu, h0 ? c[0] : c[1], 1));
}

// 96 registers a thread at launch: of 17 warps one SM quarter (16,384 registers)
// holds five.  The softmax gives some to the loaders, who keep two tiles' codes.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 88, kLoaderRegs = 104;
static_assert(kSoftmaxThreads * kSoftmaxRegs + kLoaders * kLoaderRegs + 32 * kLaunchRegs <=
                  kThreads * kLaunchRegs,
              "registers");
template <int FMT, int W>
__global__ void __launch_bounds__(kThreads, 1)
paged_mla_tc(const __nv_bfloat16* __restrict__ q_abs, PagedCache pc, BatchDev b, float scale,
             const int32_t* __restrict__ idx, const int32_t* __restrict__ n_sel, int64_t idx_width,
             int32_t rows_per_split, int32_t n_split, int32_t pair, float* __restrict__ out,
             float* __restrict__ lse, float* __restrict__ part_o, float* __restrict__ part_ml,
             int32_t* err) {
    using C = Cfg<W>;
    constexpr int kParts = W > kLatent ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t *q_full = bars, *drain = bars + 1, *s_full = bars + 2, *s_free = bars + 3,
             *p_full = bars + 4,                     // [buffer]
             *votes = bars + 24,                     // the softmax warps' votes on a tile
             *r_full = bars + 6,                     // [buffer][piece]
             *freed = bars + 16;                     // [buffer][latent block]: its values are in
    uint32_t* rinfo = reinterpret_cast<uint32_t*>(smem + C::kOffRow);
    float* l_fin = reinterpret_cast<float*>(smem + C::kOffL);
    float* m_fin = reinterpret_cast<float*>(smem + C::kOffM);
    float* inv_fin = reinterpret_cast<float*>(smem + C::kOffMs);     // output factors
    float* m_moved = reinterpret_cast<float*>(smem + C::kOffMf);     // maxima that the moved sums go by
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    uint32_t* q_max = tmem_slot + 1;
    uint32_t* raised_s = tmem_slot + 2;                              // [2] heads, a bit each
    volatile uint32_t* rows_s = tmem_slot + 5;                       // any row of the list exists
    uint32_t* far_s = tmem_slot + 4;                                 // a row past kLarge met at a raise
    // [3] tiles: the votes for a raise, and against any (16 bits each)
    volatile uint16_t* vote = reinterpret_cast<volatile uint16_t*>(tmem_slot + 8);
    uint32_t* lacking = tmem_slot + 11;                              // [2] heads without a maximum

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t q = blockIdx.y;
    const int split = blockIdx.x;
    // Two CTAs per split (gridDim.z == 2) both form the scores and divide the
    // value product and the output by latent half.
    const int half = blockIdx.z;
    const bool halved = gridDim.z == 2;
    auto owns = [&](int blk) { return !halved || (blk >> 1) == half; };
    // Two splits of a query as a cluster: each stages its output as
    // [head][latent] in its shared memory, with the log2 of its weight in m_fin
    // and whether it has rows in l_fin (all of them of logit -inf: m_fin = -inf);
    // then each combines half of the heads from
    // both through distributed shared memory.  Every thread of both CTAs calls
    // this once (an empty split with l_fin = 0).
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
        constexpr int kC4 = kLatent / 4, kEach = (kHeads / 2) * kC4 / kMergers;
        static_assert(kEach * kMergers == (kHeads / 2) * kC4, "a whole number each");
        if (threadIdx.x < kMergers) {
            // all of a thread's reads from the other CTA are in flight at once (the
            // merge takes 5 us, one after the other 8 us)
            float4 theirs[kEach];
            float f0[kEach], f1[kEach];
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int i = threadIdx.x + k * kMergers, h = (kHeads / 2) * rank + i / kC4;
                theirs[k] = st1[h * kC4 + i % kC4];
                f0[k] = m1p[h];
                f1[k] = l1p[h];
            }
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int i = threadIdx.x + k * kMergers, h = (kHeads / 2) * rank + i / kC4, c4 = i % kC4;
                const float l0 = l_fin[h], l1 = f1[k];
                // rows whose logits are all -inf: NaN weights, as of any softmax of those
                const float M = fmaxf(l0 != 0.f ? m_fin[h] : -INFINITY, l1 != 0.f ? f0[k] : -INFINITY);
                const float g0 = l0 != 0.f ? exp2f(m_fin[h] - M) : 0.f;
                const float g1 = l1 != 0.f ? exp2f(f0[k] - M) : 0.f;
                const float L = g0 + g1;
                float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
                if (L != 0.f) {
                    const float inv = 1.f / L;
                    const float4 a = l0 != 0.f ? st0[h * kC4 + c4] : r;
                    const float4 c = l1 != 0.f ? theirs[k] : r;
                    r = make_float4((a.x * g0 + c.x * g1) * inv, (a.y * g0 + c.y * g1) * inv,
                                    (a.z * g0 + c.z * g1) * inv, (a.w * g0 + c.w * g1) * inv);
                }
                o4[(q * kHeads + h) * kC4 + c4] = r;
                if (c4 == 0 && lse != nullptr)
                    lse[q * kHeads + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
            }
        }
        cl.sync();                                    // the peer's reads of this stage are done
    };

    if (threadIdx.x < kHeads) {
        m_fin[threadIdx.x] = kNoMax;
        l_fin[threadIdx.x] = 0.f;
    }
    if (threadIdx.x == 0) {
        *q_max = 0;
        *far_s = 0;
        *rows_s = 0;
        mbar_init(q_full, kSoftmaxThreads + kLoaders);
        mbar_init(drain, 1);
        mbar_init(s_full, 1);
        mbar_init(s_free, kSoftmaxThreads);
        mbar_init(votes, kSoftmaxThreads / 32);
        for (int i = 0; i < 6; ++i) vote[i] = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&p_full[i], kSoftmaxThreads);
            for (int g = 0; g < C::kPieces; ++g)      // arrivals of warps
                mbar_init(&r_full[i * C::kPieces + g], kLoaders / 32);
            for (int g = 0; g < kLatentBlocks; ++g) mbar_init(&freed[i * kLatentBlocks + g], 1);
        }
        fence_mbarrier_init();
    }
    if (warp == kMmaWarp) {
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
    // three tiles before the list's length is known (the list has idx_width).
    const bool dense = idx == nullptr;
    const int64_t j0 = (int64_t)split * rows_per_split;
    const bool loader = warp >= kSoftmaxThreads / 32 && warp < kMmaWarp;
    // loader warp lw brings the rows 8 lw .. + 7 of a tile; lane l knows where row
    // rows0 + l % 8 is
    const int rows0 = 8 * (warp - kSoftmaxThreads / 32);
    auto entry = [&](int t, int64_t end) -> int32_t {
        const int64_t j = min(j0 + (int64_t)t * kTileRows + rows0 + (lane & 7), end - 1);
        return dense ? (int32_t)j : idx[q * idx_width + j];
    };
    int32_t e0 = 0, e1 = 0, e2 = 0;
    if (loader) {
        const int64_t end = dense ? 0x7fffffff : idx_width;
        e0 = entry(0, end);
        e1 = entry(1, end);
        e2 = entry(2, end);
    }
    // The query as f16: loaded by every warp but the MMA warp, times 2^k with
    // its largest element in [2^14, 2^15), in the 128-byte swizzle.  Head
    // 32 i + 16 p + k lies in row 32 i + p + 2 k: a 16x64b load of 32 columns of
    // the scores gives a lane those of one parity, which are then 16 neighbours.
    constexpr int kQThreads = kSoftmaxThreads + kLoaders;
    constexpr int kQVecs = kHeads * W / 8;            // 16-byte vectors
    constexpr int kQPer = (kQVecs + kQThreads - 1) / kQThreads;
    auto load_query = [&](uint4 (&v)[kQPer]) {
        const uint4* src = reinterpret_cast<const uint4*>(q_abs + q * (int64_t)kHeads * W);
#pragma unroll
        for (int i = 0; i < kQPer; ++i) {
            const int c = threadIdx.x + i * kQThreads;
            v[i] = c < kQVecs ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        }
    };
    // Exponent field of the largest element, then f16 times 2^k.  2^109 makes whole
    // steps of f16 of the smallest elements there are (2^-133).
    auto query_shift = [&](uint32_t mx) -> int { return min(141 - (int)(mx >> 7), 109); };
    auto store_query = [&](const uint4 (&v)[kQPer]) {
        // the largest finite one, two at a time: with an exponent step added,
        // infinities and NaNs are negative numbers
        uint32_t two = 0x00800080u;
#pragma unroll
        for (int i = 0; i < kQPer; ++i) {
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) two = __vmaxs2(two, (u[k] & 0x7fff7fffu) + 0x00800080u);
        }
        const uint32_t mx = __reduce_max_sync(0xffffffffu, max(two & 0xffffu, two >> 16) - 0x80u);
        if (lane == 0) atomicMax(q_max, mx);
        asm volatile("bar.sync 2, %0;" ::"n"(kQThreads) : "memory");
        const float f = exp2i(query_shift(*q_max));
#pragma unroll
        for (int i = 0; i < kQPer; ++i) {
            const int c = threadIdx.x + i * kQThreads;
            if (c >= kQVecs) continue;
            const int h = c / (W / 8), c8 = c % (W / 8);
            const int n = (h & 32) + ((h >> 4) & 1) + 2 * (h & 15);
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2 x = __floats2half2_rn(__uint_as_float(u[k] << 16) * f,
                                                    __uint_as_float(u[k] & 0xffff0000u) * f);
                o[k] = *reinterpret_cast<const uint32_t*>(&x);
            }
            *reinterpret_cast<uint4*>(smem + C::kOffQ + (c8 >> 3) * kBlock + n * 128 +
                                      (((c8 & 7) ^ (n & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
    };

    // The query, and -- in a decode batch, where query q should be sequence q's --
    // the pages of the first two tiles' entries, are requested with the batch's
    // offsets rather than after them.
    uint4 qv[kQPer];
    if (warp < kMmaWarp) load_query(qv);
    const int64_t guess_row = b.n_q == b.n_seq ? q : 0;
    auto page_guess = [&](int32_t r) -> int32_t {
        const int64_t c = r >> pc.pg.shift;          // any entry of the row if r is none
        return pc.block_table[guess_row * pc.pg.table_ld + (r >= 0 && c < pc.pg.table_ld ? c : 0)];
    };
    int32_t p0 = 0, p1 = 0;
    if (loader) {
        p0 = page_guess(e0);
        p1 = page_guess(e1);
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
    const int64_t part = q * n_split + split;
    // Where this CTA's output goes, unnormalised sums of its first tiles before it
    // (a pair's outputs stay in shared memory; its sums go to the partials).
    auto sums_at = [&]() {
        return n_split == 1 ? out + q * kHeads * kLatent : part_o + part * kHeads * kLatent;
    };

    if (loader) {                                                     // ---- loads
        regs_inc<kLoaderRegs>();
        // A row's way to its codes is three dependent reads (list entry, block
        // table, codes and scales): the entries are read four tiles ahead, the
        // table three, the codes two (with the codes one ahead 970 of a tile's 4,170
        // cycles waited for them).
        // Every read is made, of some row where there is none to read, and what it
        // is worth is decided where it is used: a read within a branch is waited
        // for where the branch ends.
        const int32_t* table = pc.block_table + (int64_t)qi.seq * pc.pg.table_ld;
        auto in_list = [&](int t) { return j0 + (int64_t)t * kTileRows + rows0 + (lane & 7) < j1; };
        auto in_table = [&](int32_t r) {
            return r >= 0 && r < qi.L && (r >> pc.pg.shift) < pc.pg.table_ld;
        };
        auto page_of_row = [&](int32_t r) -> int32_t { return table[in_table(r) ? r >> pc.pg.shift : 0]; };
        // this lane's row of the warp's eight and quarter of a piece (of its 128
        // columns, or of the 64 rope columns): four lanes read 128 bytes of a row.
        // Eight lanes that store together have two rows' four quarters, of which
        // the later two take their places in another order: eight places of a line.
        const int r8 = lane >> 2, k4 = lane & 3;
        struct Tile {
            uint32_t raw[kLatentBlocks][8];          // 32 codes of each piece of row rows0 + r8
            uint4 rope;                              // 16 rope codes of the same row
            uint32_t b0, b1;                         // scales of row rows0 + lane % 8
            uint32_t has;                            // rows that exist, a bit each
        };
        auto load = [&](Tile& x, int t, int32_t r, int32_t page) {
            const bool has = in_list(t) && in_table(r) && page >= 0 && page < pc.pg.n_pages;
            const int64_t pg = has ? page : 0;
            const int64_t at = has ? (pg << pc.pg.shift) + (r & (pc.pg.page_rows - 1)) : 0;
            x.has = __ballot_sync(0xffffffffu, has);
            const uint8_t* src = pc.codes + __shfl_sync(0xffffffffu, at, r8) * W + 32 * k4;
#pragma unroll
            for (int i = 0; i < kLatentBlocks; ++i) ldg_32bytes(src + 128 * i, x.raw[i]);
            if (kParts == 2) {
                x.rope = __ldg(reinterpret_cast<const uint4*>(src + kLatent - 16 * k4));
            }
            x.b0 = __ldg(pc.scales + pg * kParts);
            x.b1 = kParts == 2 ? __ldg(pc.scales + pg * kParts + 1) : 0u;
        };
        Tile xa, xb;
        if (qi.seq != guess_row) {
            p0 = page_of_row(e0);
            p1 = page_of_row(e1);
        }
        load(xa, 0, e0, p0);
        store_query(qv);
        load(xb, 1, e1, p1);
        p0 = page_of_row(e2);
        e0 = e2;                                     // tile 2: entry and page
        e1 = entry(3, j1);
        bool ok = true;
        auto step = [&](Tile& x, int t) {
            const int buf = t & 1;
            uint8_t* rbuf = smem + C::kOffR + buf * C::kBufBytes;
            const uint32_t phase = (uint32_t)(((t >> 1) - 1) & 1);
            if (lane < 8) {
                const bool in = (x.has >> lane) & 1u;
                if (!in && in_list(t)) record_error(err, kDevBadIndex, (int32_t)q, /*where=*/34);
            }
            if (lane == 0 && x.has != 0) *rows_s = 1;    // read behind the tile's scores
            if ((x.has & 0xffu) != 0xffu) {          // zeros for rows that do not exist
                if (!((x.has >> r8) & 1u)) {
#pragma unroll
                    for (int i = 0; i < kLatentBlocks; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) x.raw[i][j] = 0;
                }
                if (!((x.has >> r8) & 1u)) x.rope = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kLatentBlocks; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a = x.raw[i][j], b = x.raw[i][4 + j];
                    x.raw[i][j] = k4 & 2 ? b : a;
                    x.raw[i][4 + j] = k4 & 2 ? a : b;
                }
#pragma unroll
            for (int i = 0; i < kLatentBlocks; ++i) {
                // the piece's columns have been read by tile t - 2's value product
                if (t >= 2 && ok) ok = warp_wait(&freed[buf * kLatentBlocks + i], phase);
                if (!ok) return;
                if (i == 0 && lane < 8)
                    rinfo[buf * kTileRows + rows0 + lane] =
                        (x.has >> lane) & 1u ? kHasRow | (x.b1 << 8) | x.b0 : 0u;
                // half of a 64-column block's line: four 16-byte places
                uint8_t* dst = rbuf + (2 * i + (k4 >> 1)) * kBlock + (rows0 + r8) * 128;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint2 lo = codes_f16<FMT>(x.raw[i][2 * j]), hi = codes_f16<FMT>(x.raw[i][2 * j + 1]);
                    *reinterpret_cast<uint4*>(dst + (((4 * (k4 & 1) + (j ^ (k4 & 2))) ^ r8) << 4)) =
                        make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&r_full[buf * C::kPieces + i]);
            }
            if constexpr (kParts == 2) {
                // the rope block held tile t - 2's W_hi, which its last product has read
                const uint2 a0 = codes_f16<FMT>(x.rope.x), a1 = codes_f16<FMT>(x.rope.y);
                const uint2 a2 = codes_f16<FMT>(x.rope.z), a3 = codes_f16<FMT>(x.rope.w);
                uint8_t* rope = rbuf + 2 * kLatentBlocks * kBlock + (rows0 + r8) * 128;
                *reinterpret_cast<uint4*>(rope + (((2 * k4) ^ r8) << 4)) = make_uint4(a0.x, a0.y, a1.x, a1.y);
                *reinterpret_cast<uint4*>(rope + (((2 * k4 + 1) ^ r8) << 4)) = make_uint4(a2.x, a2.y, a3.x, a3.y);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&r_full[buf * C::kPieces + kLatentBlocks]);
            }
            // the codes last: a wait for a load can be one for newer loads too
            const int32_t r = e0, page = p0;
            p0 = page_of_row(e1);
            e0 = e1;
            e1 = entry(t + 4, j1);
            load(x, t + 2, r, page);
        };
        for (int t = 0; t < n_tiles && ok; t += 2) {
            step(xa, t);
            if (t + 1 < n_tiles && ok) step(xb, t + 1);
        }
        if (!ok && threadIdx.x == kSoftmaxThreads) record_error(err, kDevTimeout, (int32_t)q, /*where=*/35);
    } else if (warp == kMmaWarp) {                                    // ---- MMA issue
        if (elect_one()) {
            constexpr uint32_t idesc_s = idesc_f16_f32_major(kTileRows, kHeads, 0, 0);
            constexpr uint32_t idesc_pv = idesc_f16_f32_major(128, kHeads, 1, 1);
            constexpr uint32_t idesc_pv2 = idesc_f16_f32_major(128, 2 * kHeads, 1, 1);
            const uint32_t base = smem_u32(smem);
            const uint64_t d_q = sdesc_kmajor_sw128(base + C::kOffQ);
            bool ok = mbar_wait(q_full, 0, kWaitNs);
            // Whatever is ready is issued: a tile's scores, from its first piece on
            // (in straight line: the compiler keeps the descriptors in uniform
            // registers only there), and the values of the tile whose weights are in.
            int next_s = 0, next_v = 0;
            uint32_t idle = 0;
            uint64_t t_prog = 0;
            while (ok && next_v < n_tiles) {
                bool progressed = false;
                if (next_s < n_tiles && next_s <= next_v + 1 &&
                    mbar_test_wait(&r_full[(next_s & 1) * C::kPieces], (uint32_t)((next_s >> 1) & 1)) &&
                    (next_s == 0 || mbar_test_wait(s_free, (uint32_t)((next_s - 1) & 1)))) {
                    // S^T(s) = R(s) Q^T
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
                            const bool rope = cb >= kLatent / 64;
                            mma_bf16_ss(tmem_base + (rope ? kSRopeCol : kSCol), d_r + o, d_q + o, idesc_s,
                                        kk != 0 || (cb != 0 && !rope) ? 1u : 0u);
                        }
                    }
                    mma_commit(s_full);
                    ++next_s;
                    progressed = true;
                }
                if (next_v < next_s &&
                    mbar_test_wait(&p_full[next_v & 1], (uint32_t)((next_v >> 1) & 1))) {
                    // A = R^T: MN-major, 64-column blocks 8 KB apart, 8-row
                    // groups 1 KB apart.  B = W^T: MN-major, 64 heads a block,
                    // lo's block behind hi's.
                    tc_fence_after();
                    const int bv = next_v & 1;
                    const uint32_t p_hi = base + C::off_p(bv), p_lo = base + C::kOffPlo;
                    const uint64_t d_a = sdesc_sw128(base + C::kOffR + bv * C::kBufBytes, kBlock, 1024);
                    const uint64_t d_both = sdesc_sw128(p_hi, p_lo - p_hi, 1024);
                    const uint64_t d_hi = sdesc_sw128(p_hi, 1024, 1024), d_lo = sdesc_sw128(p_lo, 1024, 1024);
                    const uint32_t acc = next_v % kFlushTiles != 0 ? 1u : 0u;
#pragma unroll
                    for (int i = 0; i < kLatentBlocks; ++i) {
                        if (owns(i)) {
#pragma unroll
                            for (int kk = 0; kk < kTileRows / 16; ++kk) {
                                const uint64_t oa = (2 * i * kBlock + kk * 2048) >> 4, ob = (kk * 2048) >> 4;
                                if (i < C::kWide) {
                                    mma_bf16_ss(tmem_base + C::o_col(i), d_a + oa, d_both + ob, idesc_pv2,
                                                kk > 0 ? 1u : acc);
                                } else {
                                    mma_bf16_ss(tmem_base + C::o_col(i), d_a + oa, d_hi + ob, idesc_pv,
                                                kk > 0 ? 1u : acc);
                                    mma_bf16_ss(tmem_base + C::o_col(i), d_a + oa, d_lo + ob, idesc_pv, 1u);
                                }
                            }
                        }
                        mma_commit(&freed[bv * kLatentBlocks + i]);
                    }
                    ++next_v;
                    progressed = true;
                }
                // the clock is slow to read: once in 256 idle rounds
                if (progressed) idle = 0;
                else if ((++idle & 255u) == 0) {
                    const uint64_t now = globaltimer_ns();
                    if (idle == 256u) t_prog = now;
                    else if (now - t_prog > kWaitNs) ok = false;
                }
            }
            if (!ok) record_error(err, kDevTimeout, (int32_t)q, /*where=*/36);
            mma_commit(drain);
            mbar_wait(drain, 0, 50000000ull);
        }
    } else {                                                          // ---- softmax
        // The scores of an M = 64 tile sit in lanes 0..15 of TMEM quadrant wq;
        // lane l of warps wq and wq + 4 takes row 16 wq + (l >> 2) + 8 (l & 1) and
        // 16 heads.
        regs_dec<kSoftmaxRegs>();
        store_query(qv);
        const int wq = warp & 3;
        const int p = (lane >> 1) & 1;
        const int srow = 16 * wq + (lane >> 2) + 8 * (lane & 1);
        const int hb = 32 * (warp >> 2) + 16 * p;    // this lane's first head
        const uint32_t lane_addr = tmem_base + ((uint32_t)(32 * wq) << 16);
        const uint32_t s_addr = lane_addr + 32 * (warp >> 2);
        // logits in log2 units, the query's power of two taken off again
        const float c2 = scale * kLog2e * exp2i(-query_shift(*q_max));
        float l_part[16];                            // sums of p over this lane's rows
#pragma unroll
        for (int e = 0; e < 16; ++e) l_part[e] = 0.f;
        constexpr int kOBlocks = kLatentBlocks + C::kWide;   // O^T's blocks of 64 columns
        float* alpha_s = l_fin;                      // rescale factors, of the sums of p in two parts
        float* alpha2_s = inv_fin;
        float m[16];                                 // the heads' running maxima
#pragma unroll
        for (int e = 0; e < 16; ++e) m[e] = kNoMax;
        bool have_max = false, far = false, ok = true;
        uint32_t vote_phase = 0;
        for (int t = 0; t < n_tiles; ++t) {
            const int bf = t & 1;
            if (ok) ok = warp_wait(s_full, (uint32_t)(t & 1));
            tc_fence_after();
            const uint32_t info = rinfo[bf * kTileRows + srow];
            const bool has = (info & kHasRow) != 0;
            const int e_row = (int)(info & 255u) - 127;
            // x = z + (e - kEBase), -inf without a row (or where z is); a factor beyond float32
            // (which multiplies zeros, or gives an infinite logit either way) is capped
            float fa = has ? c2 * e8m0(info & 255u) : 0.f;
            if (fa > 3.4028234e38f) fa = 3.4028234e38f;
            const float ev = has ? (float)(e_row - kEBase) : -INFINITY;
            const float lift = has ? fmaxf(-kLift - ev, 0.f) : 0.f;
            float x[16];                             // x[k]: head hb + k
            if constexpr (kParts == 2) {
                float fb = has ? c2 * e8m0((info >> 8) & 255u) : 0.f;
                if (fb > 3.4028234e38f) fb = 3.4028234e38f;
                float u[16];
                tmem_ld_16x64b_16_x2(s_addr + kSCol, s_addr + kSRopeCol, x, u);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = fmaf(u[e], fb, fmaf(x[e], fa, ev));
            } else {
                tmem_ld_16x64b_16(s_addr + kSCol, x);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = fmaf(x[e], fa, ev);
            }
            tc_fence_before();
            mbar_arrive(s_free);                     // the next tile's scores may be formed
            // The warps vote on whether any logit exceeds its maximum's slack, and
            // take the exponentials of the present maxima while the votes come in.
            float w[16];
            bool raise = !have_max;
            uint32_t up = 0;                         // heads whose columns of O^T follow
            if (have_max) {
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[e] -= m[e];
                    top = fmaxf(top, x[e]);
                }
                const bool any = __any_sync(0xffffffffu, top + lift > kSlack);
                // a warp of which a wait has failed votes against: all warps must meet at
                // the same barriers to the end, whatever is in the scores by then
                if (lane == 0) {
                    if (any) vote[2 * (t % 3)] = 1;
                    if (!ok) vote[1] = vote[3] = vote[5] = 1;    // for good
                    mbar_arrive(votes);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = ex2(x[e]);
                if (ok) ok = warp_wait(votes, vote_phase);
                vote_phase ^= 1u;
                const uint32_t cast = *reinterpret_cast<volatile uint32_t*>(vote + 2 * (t % 3));
                raise = ok && cast == 1u;
                // the last tile's vote, which every warp has read, for the one after next
                if (threadIdx.x == 0) vote[2 * ((t + 2) % 3)] = 0;
                if (raise) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] += m[e];
                }
            }
            if (raise) {
                const float mx = halving_max(x, lift, lane);
                if (__any_sync(0xffffffffu, has && ev > kLarge) && lane == 0) *far_s = 1;
                // in the block that W_hi takes below, free once the scores are formed
                int* red = reinterpret_cast<int*>(smem + C::off_p(bf));
                red[wq * kHeads + hb + ((lane >> 1) & 8) + ((lane >> 1) & 4) + ((lane >> 1) & 2) + (lane & 1)] =
                    fkey(mx);
                softmax_sync();
                if (threadIdx.x < kHeads) {          // raise this head's running maximum?
                    const int h = threadIdx.x;
                    const float tmax = fval(max(max(red[h], red[kHeads + h]),
                                                max(red[2 * kHeads + h], red[3 * kHeads + h])));
                    // differences, as in the vote: of logits of millions m + kSlack
                    // would round up, and a weight to f16's infinity
                    const bool up = tmax - m_fin[h] > kSlack;
                    float d = 0.f;
                    if (up) {
                        const float lower = tmax - kRoom;      // rounded, by 4 where the spacing is 8
                        const float m_new = tmax - lower > kSlack ? tmax : lower;
                        d = m_fin[h] - m_new;
                        m_fin[h] = m_new;
                    }
                    // of O^T nothing counts below 2^-120; of the sums of p, which reach
                    // from 2^127 to 2^-115, it may
                    alpha_s[h] = exp2f(fmaxf(d, -120.f));
                    alpha2_s[h] = exp2f(fminf(d + 120.f, 0.f));  // 0 from kNoMax
                    const uint32_t mask = __ballot_sync(0xffffffffu, up);
                    const uint32_t none = __ballot_sync(0xffffffffu, m_fin[h] == kNoMax);
                    if (lane == 0) {
                        raised_s[warp] = mask;
                        lacking[warp] = none;
                    }
                }
                softmax_sync();
#pragma unroll
                for (int e = 0; e < 16; ++e) l_part[e] = l_part[e] * alpha_s[hb + e] * alpha2_s[hb + e];
                far = *far_s != 0;
                // with a head that has none yet (logits of -inf so far) the next tile's
                // logits come here as they are: x - m + m would lose them
                have_max = (lacking[0] | lacking[1]) == 0;
                if (t > 0) up = raised_s[warp >> 2];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    m[e] = m_fin[hb + e];
                    x[e] -= m[e];
                    w[e] = ex2(x[e]);
                }
            }
            // w = 2^(x - m) for the values, p = w 2^-ev for their sum -- by an
            // exponential of its own (2^16 times it: the exponential ends at 2^-126)
            // where w may be below float32 and p count
            if (!far && __all_sync(0xffffffffu, !has || ev > kSmall)) {
                const float f = has ? exp2i(kEBase - e_row) : 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) l_part[e] = fmaf(w[e], f, l_part[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    l_part[e] = fmaf(has ? ex2(x[e] - ev + 16.f) : 0.f, 0x1p-16f, l_part[e]);
            }
            uint8_t* prow = smem + C::off_p(bf) + srow * 128;
            uint8_t* plow = smem + C::kOffPlo + srow * 128;
            uint32_t lo[8];
#pragma unroll
            for (int c8 = 0; c8 < 2; ++c8) {
                uint32_t hi[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = 8 * c8 + 2 * i;
                    const __half2 h2 = __floats2half2_rn(w[k], w[k + 1]);
                    const float2 hf = __half22float2(h2);
                    const __half2 l2 = __floats2half2_rn(w[k] - hf.x, w[k + 1] - hf.y);
                    hi[i] = *reinterpret_cast<const uint32_t*>(&h2);
                    lo[4 * c8 + i] = *reinterpret_cast<const uint32_t*>(&l2);
                }
                *reinterpret_cast<uint4*>(prow + ((((hb >> 3) + c8) ^ (srow & 7)) << 4)) =
                    make_uint4(hi[0], hi[1], hi[2], hi[3]);
            }
            // the previous tile's value products read W_lo
            if (t > 0 && ok)
                ok = warp_wait(&freed[((t - 1) & 1) * kLatentBlocks + kLatentBlocks - 1],
                               (uint32_t)(((t - 1) >> 1) & 1));
            // O^T, whose products so far are in (before the exponentials this held
            // them up: 3% of the time of 64 queries)
            if (up != 0) {
                tc_fence_after();
                // eight heads at a time, in each of O^T's blocks of 64 columns
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                    if (((up >> (8 * g)) & 255u) == 0) continue;
                    const int h = 32 * (warp >> 2) + 8 * g;
#pragma unroll 1
                    for (int j = 0; j < kOBlocks; j += 4) {
                        uint32_t a[4];               // the last one again past the end
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            a[i] = lane_addr + C::kOCol + 64 * min(j + i, kOBlocks - 1) + h;
                        float v[32];
                        tmem_ld_4x8cols(a, v);
#pragma unroll
                        for (int c = 0; c < 32; ++c) v[c] *= alpha_s[h + (c & 7)];
                        tmem_st_4x8cols(a, v);
                    }
                }
                tc_fence_before();
#pragma unroll
                for (int e = 0; e < 16; ++e) m[e] = m_fin[hb + e];   // not kept in registers meanwhile
            }
#pragma unroll
            for (int c8 = 0; c8 < 2; ++c8)
                *reinterpret_cast<uint4*>(plow + ((((hb >> 3) + c8) ^ (srow & 7)) << 4)) =
                    make_uint4(lo[4 * c8], lo[4 * c8 + 1], lo[4 * c8 + 2], lo[4 * c8 + 3]);
            fence_proxy_async_smem();
            if (t > 0 && t % kFlushTiles == 0) {
                // O^T moves to memory, as multiples of 2^m of the move that began a
                // head's sum, and is added to it.  Where m has grown by more than float32
                // has room for, what is there is brought to the present 2^m first.
                softmax_sync();                      // alpha_s is read
                tc_fence_after();
                if (threadIdx.x < kHeads) {
                    const int h = threadIdx.x;
                    const float grown = t == kFlushTiles ? 0.f : m_fin[h] - m_moved[h];
                    const bool anew = grown > 80.f;
                    if (anew || t == kFlushTiles) m_moved[h] = m_fin[h];
                    alpha_s[h] = anew ? 1.f : exp2f(grown);
                    alpha2_s[h] = anew ? exp2f(-grown) : 1.f;
                    const uint32_t mask = __ballot_sync(0xffffffffu, anew);
                    if (lane == 0) raised_s[warp] = mask;
                }
                softmax_sync();
                const uint32_t mask = raised_s[warp >> 2];
                float* const sums = sums_at();
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                    const int h = 32 * (warp >> 2) + 8 * g;
#pragma unroll
                    for (int j = 0; j < kOBlocks; j += 4) {
                        uint32_t a[4];               // the last one again past the end
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            a[i] = lane_addr + C::kOCol + 64 * min(j + i, kOBlocks - 1) + h;
                        float v[32];
                        tmem_ld_4x8cols(a, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int k = j + i;     // hi and lo of the wide blocks, then the others
                            const bool wide = k < 2 * C::kWide;
                            const int blk = wide ? k >> 1 : k - C::kWide;
                            if (k >= kOBlocks || (wide && (k & 1)) || !owns(blk)) continue;
                            float* dst = sums + h * kLatent + 128 * blk + 32 * wq + lane;
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                if (wide) v[8 * i + c] += v[(8 * i + c + 8) & 31];
                            if (t == kFlushTiles) {                  // a first move
#pragma unroll
                                for (int c = 0; c < 8; ++c) dst[c * kLatent] = v[8 * i + c];
                                continue;
                            }
                            if (((mask >> (8 * g)) & 255u) != 0) {  // far grown heads among these
#pragma unroll 1
                                for (int c = 0; c < 8; ++c) dst[c * kLatent] = __ldcg(dst + c * kLatent) * alpha2_s[h + c];
                            }
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                atomicAdd(dst + c * kLatent, v[8 * i + c] * alpha_s[h + c]);
                            }
                        }
                    }
                }
                tc_fence_before();
#pragma unroll
                for (int e = 0; e < 16; ++e) m[e] = m_fin[hb + e];   // not kept in registers meanwhile
            }
            tc_fence_before();
            mbar_arrive(&p_full[bf]);
        }
        {
            const int tl = n_tiles - 1;
            if (ok) ok = warp_wait(&freed[(tl & 1) * kLatentBlocks + kLatentBlocks - 1],
                                   (uint32_t)((tl >> 1) & 1));
        }
        if (!ok) record_error(err, kDevTimeout, (int32_t)q, /*where=*/37);
        // row sums to shared memory (the row buffers are free now)
        float* lsc = reinterpret_cast<float*>(smem + C::kOffR);
#pragma unroll
        for (int e = 0; e < 16; ++e) lsc[srow * (kHeads + 1) + hb + e] = l_part[e];
        softmax_sync();
        if (threadIdx.x < kHeads) {
            // the head's weight: out = O^T 2^kEBase / l, log2 of it m + log2 l
            const int h = threadIdx.x;
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int r = 0; r < kTileRows; ++r) s4[r & 3] += lsc[r * (kHeads + 1) + h];
            const float l = (s4[0] + s4[1]) + (s4[2] + s4[3]);
            m_moved[h] = exp2f(m_moved[h] - m_fin[h]);       // what the moved sums are worth
            if (l != 0.f) {
                inv_fin[h] = exp2i(kEBase) / l;
                m_fin[h] += log2f(l);
            } else {
                // no rows, or rows of logit -inf only: NaN unless another split has more
                const bool rows = *rows_s != 0, nan = rows && n_split == 1;
                inv_fin[h] = nan ? NAN : 0.f;
                m_fin[h] = nan ? NAN : rows ? -INFINITY : kNoMax;
            }
            l_fin[h] = l != 0.f || *rows_s != 0 ? 1.f : 0.f;
        }
    }

    // ---- epilogue, warps 0-15: O^T read out of TMEM, times 2^kEBase / l
    if (warp < kMmaWarp) {
        asm volatile("bar.sync 3, %0;" ::"n"(kMergers) : "memory");
        tc_fence_after();
        const int wq = warp & 3, hb = 16 * (warp >> 2);      // this warp's heads
        const uint32_t lane_addr = tmem_base + ((uint32_t)(32 * wq) << 16);
        const bool final_out = n_split == 1, moved = n_tiles > kFlushTiles;
        float* const sums = sums_at();
        float* dst = pair ? stage : sums;
        float inv[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) inv[e] = inv_fin[hb + e];
        // lane 32 wq + lane of block i holds latent column 128 i + 32 wq + lane
#pragma unroll
        for (int i = 0; i < kLatentBlocks; ++i) {
            if (!owns(i)) continue;
            const int c = 128 * i + 32 * wq + lane;
            float v[16];
            if (i < C::kWide) {                      // hi and lo halves
                float u[16];
                tmem_ld_16cols_x2(lane_addr + C::o_col(i) + hb, lane_addr + C::o_col(i) + 64 + hb, v, u);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] += u[e];
            } else {
                tmem_ld_16cols(lane_addr + C::o_col(i) + hb, v);
            }
            if (moved) {
                float u[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] = __ldcg(sums + (hb + e) * kLatent + c);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = fmaf(u[e], m_moved[hb + e], v[e]);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) dst[(hb + e) * kLatent + c] = v[e] * inv[e];
        }
        if (threadIdx.x < kHeads && !pair && half == 0) {
            const int h = threadIdx.x;
            const float l = l_fin[h], m = l == 0.f ? -INFINITY : m_fin[h] * kLn2;
            if (final_out) {
                if (lse != nullptr) lse[q * kHeads + h] = m;
            } else {
                // NaN as a sum: the merge takes its maximum over numbers
                part_ml[(part * kHeads + h) * 2] = m == m ? m : 0.f;
                part_ml[(part * kHeads + h) * 2 + 1] = m == m ? l : m;
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
    e = cudaLaunchKernelEx(&cfg, kern, static_cast<const __nv_bfloat16*>(q_abs), pc, b, sh.scale, idx, n_sel, sh.index_row_width(), rps,
                           n_split, pair, out, lse, part_o, part_ml, err);
    if (e != cudaSuccess || n_split <= 2) return e;
    return launch_merge_splits(b.n_q, n_split, part_o, part_ml, out, lse, st, /*nan_lse=*/true);
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
