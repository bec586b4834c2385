// expand_kv_tc.cu -- latent rows into every head's keys and values on the tcgen05
// tensor cores (bf16): [n_rows, 512] times [heads * d, 512]^T, for w_uk and w_uv in one launch.
//
// A pair of CTAs (cta_group::2) computes tiles of 256 rows by NT features, each CTA with
// 128 of the rows and half of the features to load.  Its tiles are neighbours along
// the features, so the rows stay in shared memory (128 KB a CTA) and only
// weights stream, out of L2: 32 bytes a cycle and CTA at NT = 256, where the products read
// another 64 of the 128 that shared memory has.  Two accumulators in TMEM, so that a
// tile's output is written beside the next one's products.  In each CTA
//   warp 4    TMA: the rows in eight blocks of 64 columns, a block again as soon as the
//             last tile of the rows before has read it; a ring of weight blocks;
//   warp 5    in the first CTA issues the products for both;
//   warps 0-3 epilogue, a row to a thread: bf16 in whole sectors.
// Bound by writing for prompts: 4,096 rows are 235 MB of keys and values, 63 us at the
// rate of 3.7 TB/s at which this memory takes writes alone; without the stores the
// products take 56 us.  A few rows: by reading the weights (29 MB).
#include "dsa_kernels.cuh"
#include "pair.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kM = 256, kRows = 128;                     // rows of a tile and of a CTA
constexpr int kDepth = 512, kKB = kDepth / 64;           // the sum, in blocks of 64
constexpr uint32_t kABlock = kRows * 128;
template <int NT>
constexpr int kRing = NT == 256 ? 6 : 12;                // weight blocks: 96 KB of them
constexpr int kThreads = 192;
constexpr int kTmaWarp = 4, kMmaWarp = 5;
constexpr uint32_t kBarBytes = 1024;

struct Shared {
    uint64_t a_full[kKB], a_free[kKB], full[12], empty[12], acc_full[2], acc_free[2], drain;
    uint32_t tmem;
    int32_t abort;
};
static_assert(sizeof(Shared) <= kBarBytes, "barriers");

template <int NT>
constexpr uint32_t kSmem = 1024 + kBarBytes + kKB * kABlock + kRing<NT> * (NT / 2) * 128;

template <int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
expand_tc(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_uk,
          const __grid_constant__ CUtensorMap tm_uv, __nv_bfloat16* __restrict__ k_nope,
          __nv_bfloat16* __restrict__ v, const int64_t n_rows, const int32_t n_k, const int32_t n_v,
          const int32_t box_rows, int32_t* err) {
    constexpr uint32_t kBBlock = NT / 2 * 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Shared& s = *reinterpret_cast<Shared*>(smem);
    uint8_t* As = smem + kBarBytes;
    uint8_t* Bs = As + kKB * kABlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int64_t n_tiles = (n_k + n_v) / NT, total = (n_rows + kM - 1) / kM * n_tiles;
    const int64_t pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const int64_t begin = total * pair / pairs, end = total * (pair + 1) / pairs;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kKB; ++i) {
            mbar_init(&s.a_full[i], 1);
            mbar_init(&s.a_free[i], 1);
        }
        for (int i = 0; i < kRing<NT>; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_free[i], 2 * kRows / 32);
        }
        mbar_init(&s.drain, 1);
        s.abort = 0;
        fence_mbarrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(&s.tmem, 2 * NT);
        tmem_relinquish_pair();
    }
    if (warp == kTmaWarp && lane == 0) {
        prefetch_tensormap(&tm_rows);
        prefetch_tensormap(&tm_uk);
        prefetch_tensormap(&tm_uv);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int32_t* abort = &s.abort;
    pdl_wait();
    pdl_trigger();

    if (warp == kTmaWarp) {
        if (lane == 0) {                                           // ---- TMA
            bool ok = true;
            Place p;
            int64_t m = begin / n_tiles;
            int n = (int)(begin % n_tiles), loads = 0;             // loads: of rows so far
            for (int64_t u = begin; u < end && ok; ++u) {
                const bool fresh = u == begin || n == 0;
                const bool is_v = (int64_t)n * NT >= n_k;
                const int32_t y = (is_v ? n * NT - n_k : n * NT) + (int32_t)rank * (NT / 2);
                for (int kb = 0; kb < kKB; ++kb) {
                    if (fresh) {
                        ok = loads == 0 || wait(&s.a_free[kb], (loads - 1) & 1, abort);
                        if (!ok) break;
                        if (rank == 0) mbar_arrive_expect_tx(&s.a_full[kb], 2 * box_rows * 128);
                        tma_load_2d_pair(As + kb * kABlock, &tm_rows, cluster_addr(&s.a_full[kb], 0), kb * 64,
                                         (int32_t)(m * kM + rank * kRows));
                    }
                    ok = wait(&s.empty[p.at], p.parity ^ 1, abort);
                    if (!ok) break;
                    if (rank == 0) mbar_arrive_expect_tx(&s.full[p.at], 2 * kBBlock);
                    tma_load_2d_pair(Bs + p.at * kBBlock, is_v ? &tm_uv : &tm_uk, cluster_addr(&s.full[p.at], 0),
                                     kb * 64, y);
                    p.step(kRing<NT>);
                }
                if (fresh) ++loads;
                if (++n == n_tiles) { n = 0; ++m; }
            }
            if (!ok) {
                record_error(err, kDevTimeout, blockIdx.x, 70);
                *abort = 1;
                // copies in flight land first: their barriers are the first CTA's
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 50000000ull) {}
            }
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0 && elect_one()) {                            // ---- products
            bool ok = true;
            Place p;
            const uint32_t a_addr = smem_u32(As), b_addr = smem_u32(Bs), idesc = idesc_bf16_f32(kM, NT);
            int64_t n = begin % n_tiles;
            int loads = 0, t = 0;
            for (int64_t u = begin; u < end && ok; ++u, ++t) {
                const bool fresh = u == begin || n == 0, last = u + 1 == end || n + 1 == n_tiles;
                const uint32_t d = tmem + (t & 1) * NT;
                ok = t < 2 || wait(&s.acc_free[t & 1], ((t >> 1) - 1) & 1, abort);
                for (int kb = 0; kb < kKB; ++kb) {
                    ok = ok && (!fresh || wait(&s.a_full[kb], loads & 1, abort)) && wait(&s.full[p.at], p.parity, abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ss_pair(d, sdesc_kmajor_sw128(a_addr + kb * kABlock + kk * 32),
                                         sdesc_kmajor_sw128(b_addr + p.at * kBBlock + kk * 32), idesc, (kb | kk) != 0);
                    mma_commit_pair(&s.empty[p.at]);
                    if (last) mma_commit_pair(&s.a_free[kb]);
                    p.step(kRing<NT>);
                }
                if (ok) mma_commit_pair(&s.acc_full[t & 1]);
                if (fresh) ++loads;
                if (++n == n_tiles) n = 0;
            }
            if (!ok) {
                record_error(err, kDevTimeout, blockIdx.x, 71);
                *abort = 1;
                mma_commit_pair(&s.drain);                         // every issued product retired
                mbar_wait(&s.drain, 0, 50000000ull);
            }
        }
        __syncwarp();
    } else {                                                       // ---- epilogue
        const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
        bool ok = true;
        int t = 0;
        int64_t m = begin / n_tiles;
        int n = (int)(begin % n_tiles);
        for (int64_t u = begin; u < end; ++u, ++t) {
            ok = warp_wait(&s.acc_full[t & 1], (t >> 1) & 1, abort);
            if (!ok) break;
            tc_fence_after();
            const int64_t row = m * kM + rank * kRows + threadIdx.x;
            const bool is_v = (int64_t)n * NT >= n_k, mine = row < n_rows;
            __nv_bfloat16* out = is_v ? v + row * n_v + (n * NT - n_k) : k_nope + row * n_k + n * NT;
#pragma unroll
            for (int c = 0; c < NT; c += 64) {
                float o[2][32];
                tmem_ld_32cols_x2(lane_addr + (t & 1) * NT + c, lane_addr + (t & 1) * NT + c + 32, o[0], o[1]);
                if (c + 64 == NT) {                                // the accumulator may be written again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(cluster_addr(&s.acc_free[t & 1], 0));
                }
                if (!mine) continue;
#pragma unroll
                for (int e = 0; e < 64; e += 16) {
                    uint32_t x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = pack(o[e >> 5][(e & 31) + 2 * i], o[e >> 5][(e & 31) + 2 * i + 1]);
                    store_sector(out + c + e, x);
                }
            }
            if (++n == n_tiles) { n = 0; ++m; }
        }
        if (!ok) {
            if (lane == 0) record_error(err, kDevTimeout, blockIdx.x, 72);
            *abort = 1;
        }
    }
    // neither CTA leaves while the other's products or signals still reach it
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 2 * NT);
    }
}

template <int NT>
cudaError_t launch(const Shape& sh, int64_t n_rows, int32_t n_k, int32_t n_v, const void* rows, const void* w_uk,
                   const void* w_uv, void* k_nope, void* v, int32_t* err, cudaStream_t st) {
    CUtensorMap tr, tk, tv;
    auto map = [](CUtensorMap* m, const void* base, int64_t n, int64_t width, uint32_t box) {
        const uint64_t dims[2] = {(uint64_t)kDepth, (uint64_t)n}, strides[1] = {(uint64_t)width * 2};
        const uint32_t b[2] = {64, box};
        return encode_bf16_map(m, base, 2, dims, strides, b);
    };
    // few rows: no more of a tile is loaded (its other rows' results are not stored)
    const int32_t box_rows = n_rows < kRows ? (int32_t)(n_rows + 7) / 8 * 8 : kRows;
    if (!map(&tr, rows, n_rows, sh.width(), box_rows) || !map(&tk, w_uk, n_k, kDepth, NT / 2) ||
        !map(&tv, w_uv, n_v, kDepth, NT / 2))
        return cudaErrorInvalidValue;
    auto kern = expand_tc<NT>;
    cudaError_t e = ensure_dyn_smem((const void*)kern, (int)kSmem<NT>);
    if (e != cudaSuccess) return e;
    const int64_t total = (n_rows + kM - 1) / kM * ((n_k + n_v) / NT);
    int64_t pairs = sm_count() / 2;
    if (pairs > total) pairs = total;
    return launch_pdl(kern, dim3((unsigned)(2 * pairs)), dim3(kThreads), kSmem<NT>, st, tr, tk, tv,
                      static_cast<__nv_bfloat16*>(k_nope), static_cast<__nv_bfloat16*>(v), n_rows, n_k, n_v, box_rows, err);
}

}  // namespace

cudaError_t launch_expand_tc(const Shape& sh, int64_t n_rows, int32_t nope, int32_t v_dim, const void* rows,
                             const void* w_uk, const void* w_uv, void* k_nope, void* v, int32_t* err,
                             cudaStream_t st) {
    const int32_t n_k = sh.heads * nope, n_v = sh.heads * v_dim;
    // tiles of 128 features where the pair with the most has less to do with them
    // than with tiles of 256: few rows
    const int64_t pairs = sm_count() / 2, wide = (n_rows + kM - 1) / kM * ((n_k + n_v) / 256);
    const bool narrow = (2 * wide + pairs - 1) / pairs < 2 * ((wide + pairs - 1) / pairs) && wide < 4 * pairs;
    return narrow ? launch<128>(sh, n_rows, n_k, n_v, rows, w_uk, w_uv, k_nope, v, err, st)
                  : launch<256>(sh, n_rows, n_k, n_v, rows, w_uk, w_uv, k_nope, v, err, st);
}

}  // namespace dsa
