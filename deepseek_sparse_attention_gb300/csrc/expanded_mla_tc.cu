// expanded_mla_tc.cu -- causal attention over expanded keys and values on the
// tcgen05 tensor cores (bf16).
//
//   S = Q K^T (M = 256 queries, N = 128 keys, K = the head's width), one pass over
//   the key tiles with a running maximum, O += P V (M = 256, N = v_dim, K = 128 keys)
//
// A pair of CTAs (cta_group::2) per (tile of 256 queries, head, split of the key
// tiles): each has 128 of the queries, their S, P and O, and loads half of the keys'
// rows and half of the values' columns.  In each CTA
//   warp 8     TMA: the queries once, then a ring of units in the order of their use:
//              a tile's keys (columns in blocks of 64, the rope block from the cache rows,
//              for every head), a tile's values.  (Handed over in eight blocks of 8 KB a
//              tile, with or without a pair, a tile took 3,700 cycles: the threads that
//              issue copies and products spend some 200 on each hand-over.)
//   warp 9     in the first CTA issues the products for both, S of tile t + 1 before O
//              of tile t;
//   warps 0-7  softmax, a query row and half of its keys to a thread: S from TMEM,
//              exp, P in bf16 back over S (O takes it from TMEM as its A operand).
//              Row maxima are raised only when a logit exceeds them by more than
//              kSlack, so the two halves of a row share a maximum without telling each
//              other theirs: a barrier that also votes says whether any row is raised,
//              and only then they are exchanged and O is rescaled in TMEM;
//   warps 10-11 values of tiles that some query sees only in part: NaN and infinities
//              are taken out of shared memory (0 times either is NaN) and given back in the
//              epilogue to the queries that see them.
// P is rounded to bf16 because both operands of the value product have one
// type and V is bf16: 2^-8 of a weight at most, of random sign.
#include <math.h>

#include "expanded_mla.cuh"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kQ = kExpandedTcQ, kK = kExpandedTcK;      // queries and keys of a tile
constexpr int kRows = kQ / 2;                            // queries of a CTA
constexpr uint32_t kQBlock = kRows * 128;                // 64 columns of them
constexpr uint32_t kKBlock = kK / 2 * 128;               // 64 columns of a CTA's half of a tile's keys
constexpr int kMaxRing = 14;
constexpr int kSoftmax = 256;                            // threads
constexpr int kTmaWarp = 8, kMmaWarp = 9, kCleanWarp = 10;
constexpr int kThreads = 384;
constexpr int kCleaners = 64;
constexpr uint32_t kOCol = 256, kTmemCols = 512;         // S0, S1 at 0 and 128
constexpr uint32_t kSmem = 227 * 1024;
constexpr uint32_t kBarBytes = 2048;
constexpr long long kWaitCycles = 4000000000ll;          // about 2 s
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;                            // weights stay below 2^8

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

struct Bars {
    uint64_t full[kMaxRing], empty[kMaxRing], part[kMaxRing], clean[kMaxRing];
    uint64_t q_full, s_full[2], p_full[2], o_done, o_last, drain;
    float half[kSoftmax];                                // maxima, then sums, of a row's halves
    uint32_t tmem;
    int32_t abort, poison;
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers");

// Two at a time: x * a + b, and sums.
__device__ __forceinline__ float2 fma_x2(float2 x, float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, a, b, d;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 a, {%4, %5};\n\tmov.b64 b, {%6, %7};\n\t"
        "fma.rn.f32x2 d, x, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add_x2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The softmax warps meet here, and learn whether any thread's `p` holds.
__device__ __forceinline__ bool softmax_vote(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)p)
        : "memory");
    return r != 0;
}

// A place in the ring and the parity of its use, one block after the other.
struct Place {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void step(int ring) {
        if (++at == ring) { at = 0; parity ^= 1; }
    }
};

// A wait that ends early when another role gave up.  The clock is the SM's: reading
// the global timer between two tries cost up to 2,000 cycles after the arrival.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (*abort != 0 || clock64() - t0 > kWaitCycles) return false;
    return true;
}
// The same made by a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort) {
    return __all_sync(0xffffffffu, wait(bar, parity, abort));
}

// Room for either kind of unit.
__host__ __device__ constexpr uint32_t unit_size(int nk, int v_dim) {
    const uint32_t k = nk * kKBlock, v = v_dim / 128 * (kK * 128);
    return k > v ? k : v;
}

template <int VD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
expanded_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
            const ExpandedArgs a, const int32_t slots, const int32_t ring) {
    constexpr uint32_t kVBlock = kK * 128;               // 64 columns of a tile's values
    constexpr uint32_t kVBytes = VD / 128 * kVBlock;     // a CTA's half of them
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Bars& s = *reinterpret_cast<Bars*>(smem);
    uint8_t* Qs = smem + kBarBytes;
    const int nk = (a.nope + a.rope) / 64, nope_blocks = a.nope / 64;   // blocks of a tile's keys
    const uint32_t unit_bytes = unit_size(nk, VD);       // of the ring
    uint8_t* Rs = Qs + nk * kQBlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a head's tiles one after the other (its keys and values stay in L2), the
    // longest first
    const uint32_t unit = blockIdx.x / 2, rank = cluster_rank();
    const int split = (int)(unit % a.n_split);
    const int64_t slot = slots - 1 - (int64_t)(unit / a.n_split) % slots;
    const int h = (int)(unit / a.n_split / slots);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxRing; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
            mbar_init(&s.part[i], 1);
            mbar_init(&s.clean[i], 2 * kCleaners / 32);
        }
        mbar_init(&s.q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 2 * kSoftmax / 32);
        }
        mbar_init(&s.o_done, 1);
        mbar_init(&s.o_last, 1);
        mbar_init(&s.drain, 1);
        s.abort = 0;
        s.poison = 0;
        fence_mbarrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(&s.tmem, kTmemCols);
        tmem_relinquish_pair();
    }
    if (warp == kTmaWarp && lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_r);
        prefetch_tensormap(&tm_v);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int32_t* abort = &s.abort;
    pdl_wait();
    pdl_trigger();
    ExpandedTile t;
    const bool live = expanded_tile(a.b, slot, split, a.n_split, kQ, kK, threadIdx.x == 0 ? a.err : nullptr, 61, t);
    const int n = live ? t.kt1 - t.kt0 : 0;
    // key tiles from this one on are not seen in full by every query
    const int partial = live ? (int)(t.first / kK) : 0;

    if (n > 0 && warp == kTmaWarp) {
        if (lane == 0) {                                           // ---- TMA
            bool ok = true;
            Place p;
            // A unit of both CTAs counts on the first one's barrier -- or, of values that
            // the cleaners see first, on each CTA's own, and the full barrier's phase passes.
            auto next = [&](uint32_t bytes, uint32_t& bar, bool partly) -> uint8_t* {
                ok = wait(&s.empty[p.at], p.parity ^ 1, abort);
                if (!ok) return nullptr;
                uint8_t* dst = Rs + p.at * unit_bytes;
                if (partly) {
                    bar = smem_u32(&s.part[p.at]);
                    mbar_arrive_expect_tx(&s.part[p.at], bytes);
                    if (rank == 0) mbar_arrive(&s.full[p.at]);
                } else {
                    bar = cluster_addr(&s.full[p.at], 0);
                    if (rank == 0) mbar_arrive_expect_tx(&s.full[p.at], 2 * bytes);
                }
                p.step(ring);
                return dst;
            };
            auto keys = [&](int kt) {                              // half of the tile's rows
                const int32_t y = (int32_t)(t.row0 + (int64_t)kt * kK + rank * (kK / 2));
                uint32_t bar;
                uint8_t* dst = next(nk * kKBlock, bar, false);
                for (int b = 0; b < nk && ok; ++b) {
                    if (b < nope_blocks) tma_load_3d_pair(dst + b * kKBlock, &tm_k, bar, b * 64, h, y);
                    else tma_load_2d_pair(dst + b * kKBlock, &tm_r, bar, a.kv_lora + (b - nope_blocks) * 64, y);
                }
            };
            auto values = [&](int kt) {                            // half of the columns
                const int32_t y = (int32_t)(t.row0 + (int64_t)kt * kK);
                uint32_t bar;
                uint8_t* dst = next(kVBytes, bar, kt >= partial);
                for (int c = 0; c < VD / 128 && ok; ++c)
                    tma_load_3d_pair(dst + c * kVBlock, &tm_v, bar, rank * (VD / 2) + c * 64, h, y);
            };
            if (rank == 0) mbar_arrive_expect_tx(&s.q_full, 2 * nk * kQBlock);
            for (int b = 0; b < nk; ++b)
                tma_load_3d_pair(Qs + b * kQBlock, &tm_q, cluster_addr(&s.q_full, 0), b * 64, h,
                                 (int32_t)(t.q0 + rank * kRows));
            keys(t.kt0);
            for (int i = 0; i < n && ok; ++i) {
                if (i + 1 < n) keys(t.kt0 + i + 1);
                if (ok) values(t.kt0 + i);
            }
            if (!ok) {
                record_error(a.err, kDevTimeout, blockIdx.x, 62);
                *abort = 1;
                // copies in flight land first: their barriers are partly the other CTA's
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 50000000ull) {}
            }
        }
    } else if (n > 0 && warp == kMmaWarp && rank == 0) {
        if (elect_one()) {                                         // ---- products
            bool ok = wait(&s.q_full, 0, abort);
            Place p;
            uint32_t cleaned = 0;                                  // parities of the clean barriers
            const uint32_t q_addr = smem_u32(Qs), r_addr = smem_u32(Rs);
            const uint32_t id_s = idesc_bf16_f32(kQ, kK), id_o = idesc_bf16_f32_major(kQ, VD, 0, 1);
            auto scores = [&](int i) {
                ok = ok && wait(&s.full[p.at], p.parity, abort);
                if (!ok) return;
                tc_fence_after();
                const uint32_t k_addr = r_addr + p.at * unit_bytes, d = tmem + (i & 1) * kK;
                for (int b = 0; b < nk; ++b) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ss_pair(d, sdesc_kmajor_sw128(q_addr + b * kQBlock + kk * 32),
                                         sdesc_kmajor_sw128(k_addr + b * kKBlock + kk * 32), id_s, (b | kk) != 0);
                }
                mma_commit_pair(&s.empty[p.at]);
                mma_commit_pair(&s.s_full[i & 1]);
                p.step(ring);
            };
            auto values = [&](int i) {
                ok = wait(&s.full[p.at], p.parity, abort);
                if (ok && t.kt0 + i >= partial) {
                    ok = wait(&s.clean[p.at], (cleaned >> p.at) & 1, abort);
                    cleaned ^= 1u << p.at;
                }
                ok = ok && wait(&s.p_full[i & 1], (i >> 1) & 1, abort);
                if (!ok) return;
                tc_fence_after();
                const uint32_t v_addr = r_addr + p.at * unit_bytes, w = tmem + (i & 1) * kK;
#pragma unroll
                for (int kk = 0; kk < kK / 16; ++kk)
                    mma_bf16_ts_pair(tmem + kOCol, w + kk * 8, sdesc_sw128(v_addr + kk * 2048, kVBlock, 1024), id_o,
                                     (i | kk) != 0);
                mma_commit_pair(&s.empty[p.at]);
                mma_commit_pair(&s.o_done);
                p.step(ring);
            };
            scores(0);
            for (int i = 0; i < n && ok; ++i) {
                if (i + 1 < n) scores(i + 1);
                if (ok) values(i);
            }
            if (ok) {
                mma_commit_pair(&s.o_last);
            } else {
                record_error(a.err, kDevTimeout, blockIdx.x, 63);
                *abort = 1;
                mma_commit_pair(&s.drain);                         // every issued product retired
                mbar_wait(&s.drain, 0, 50000000ull);
            }
        }
        __syncwarp();
    } else if (n > 0 && warp >= kCleanWarp) {                      // ---- hidden values
        const int c = threadIdx.x - kCleanWarp * 32;
        uint32_t parted = 0;                                       // parities of the part barriers
        for (int i = partial > t.kt0 ? partial - t.kt0 : 0; i < n; ++i) {
            // units used before tile i's values: keys of tiles 0 .. min(i + 1, n - 1), values of 0 .. i - 1
            const uint32_t at = (uint32_t)((i + 1 < n ? i + 2 : n) + i) % ring;
            const bool ok = warp_wait(&s.part[at], (parted >> at) & 1, abort);
            parted ^= 1u << at;
            if (!ok) {
                if (lane == 0) record_error(a.err, kDevTimeout, blockIdx.x, 64);
                *abort = 1;
                break;
            }
            uint4* p = reinterpret_cast<uint4*>(Rs + at * unit_bytes) + c;
            // an exponent of ones carries into its half's sign
            auto odd = [](uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
            bool bad = false;
#pragma unroll 1
            for (int k = 0; k < (int)(kVBytes / 16 / kCleaners); k += 8) {
                uint4 x[8];
                uint32_t any = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = p[(k + e) * kCleaners];
#pragma unroll
                for (int e = 0; e < 8; ++e) any |= odd(x[e].x) | odd(x[e].y) | odd(x[e].z) | odd(x[e].w);
                if (any == 0) continue;
                bad = true;
                // the halves that are odd become zeros
                auto clean = [&](uint32_t w) { const uint32_t m = odd(w) >> 15; return w & ~(m * 0xffffu); };
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    p[(k + e) * kCleaners] = make_uint4(clean(x[e].x), clean(x[e].y), clean(x[e].z), clean(x[e].w));
            }
            if (bad) {                                             // both CTAs give them back
                *(volatile int32_t*)&s.poison = 1;
                st_cluster(cluster_addr(&s.poison, rank ^ 1), 1);
                fence_cluster();
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_addr(&s.clean[at], 0));
        }
    } else if (warp < kSoftmax / 32 && live) {                     // ---- softmax
        const int mine_row = threadIdx.x & 127, half = threadIdx.x >> 7;
        const int row = (int)rank * kRows + mine_row;              // of the pair's queries
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float scale = a.scale * kLog2e;
        const int64_t sees = t.first + row;
        float m = -INFINITY, l = 0.f;                              // l: of this half's keys
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            // a warp that gives up votes and meets the others all the same
            ok = ok && warp_wait(&s.s_full[i & 1], (i >> 1) & 1, abort);
            tc_fence_after();
            const uint32_t at = lane_addr + (i & 1) * kK;
            float v[2][32];
            tmem_ld_32cols_x2(at + half * 64, at + half * 64 + 32, v[0], v[1]);
            if (t.kt0 + i >= partial) {
                // this half's keys of the tile that the row sees
                const int64_t left = sees - (int64_t)(t.kt0 + i) * kK - half * 64;
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (e >= left) v[e >> 5][e & 31] = -INFINITY;
            }
            float tops[4] = {v[0][0], v[0][1], v[0][2], v[0][3]};
#pragma unroll
            for (int e = 4; e < 64; ++e) tops[e & 3] = fmaxf(tops[e & 3], v[e >> 5][e & 31]);
            float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale;
            // of -inf: any logit above it
            if (softmax_vote(top > m + kSlack || !ok)) {
                s.half[threadIdx.x] = top;
                ok = !softmax_vote(!ok);                           // all go on, or none
                if (!ok) break;
                top = fmaxf(top, s.half[threadIdx.x ^ 128]);
                const float mn = top > m + kSlack ? top : m;
                const float f = mn == m ? 1.f : ex2(m - mn);
                if (__any_sync(0xffffffffu, mn != m) && i > 0) {
                    ok = warp_wait(&s.o_done, (i - 1) & 1, abort);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = half * (VD / 2); c < (half + 1) * (VD / 2) && ok; c += 32) {
                        float o[32];
                        tmem_ld_32cols(lane_addr + kOCol + c, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tmem_st_32cols(lane_addr + kOCol + c, o);
                    }
                }
                l *= f;
                m = mn;
                softmax_vote(false);                               // maxima read: free to be written
            }
            const float base = m == -INFINITY ? 0.f : -m;          // no logit above -inf yet
            const float2 scale2 = make_float2(scale, scale), base2 = make_float2(base, base);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            float w[32];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
                float2 p = fma_x2(make_float2(v[e >> 5][e & 31], v[e >> 5][(e & 31) + 1]), scale2, base2);
                p.x = ex2(p.x);
                p.y = ex2(p.y);
                sum[(e >> 1) & 1] = add_x2(sum[(e >> 1) & 1], p);
                w[e >> 1] = __uint_as_float(pack(p.x, p.y));
            }
            tmem_st_32cols(at + half * 32, w);
            const float2 both = add_x2(sum[0], sum[1]);
            l += both.x + both.y;
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive_cluster(cluster_addr(&s.p_full[i & 1], 0));
        }
        s.half[threadIdx.x] = l;
        ok = ok && (n == 0 || warp_wait(&s.o_last, 0, abort));
        ok = !softmax_vote(!ok);
        if (!ok) {
            if (lane == 0) record_error(a.err, kDevTimeout, blockIdx.x, 65);
            *abort = 1;
        } else {
            tc_fence_after();
            l += s.half[threadIdx.x ^ 128];
            const int64_t qh = (t.q0 + row) * a.heads + h;
            const bool mine = row < t.n_q;
            const bool poison = n > 0 && *(volatile int32_t*)&s.poison != 0;
            const float inv = 1.f / l;
            if (a.n_split > 1 && mine && half == 0)
                *reinterpret_cast<float2*>(a.part_ml + (qh * a.n_split + split) * 2) = make_float2(m, l);
            if (a.n_split == 1 && mine && half == 0 && a.lse != nullptr) a.lse[qh] = expanded_lse(m, l);
            const int64_t from = (int64_t)(partial > t.kt0 ? partial : t.kt0) * kK;
            const int64_t to = sees < (int64_t)t.kt1 * kK ? sees : (int64_t)t.kt1 * kK;
#pragma unroll 1
            for (int c = half * (VD / 2); c < (half + 1) * (VD / 2) && n > 0; c += 32) {
                float o[32];
                tmem_ld_32cols(lane_addr + kOCol + c, o);
                if (poison && mine) {
                    for (int64_t j = from; j < to; ++j) {
                        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.v) +
                                                 ((t.row0 + j) * a.heads + h) * VD + c;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float y = __bfloat162float(x[e]);
                            if (!isfinite(y)) o[e] += y;
                        }
                    }
                }
                if (!mine) continue;
                if (a.n_split > 1) {
                    float4* p = reinterpret_cast<float4*>(a.part_o + (qh * a.n_split + split) * VD + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        p[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                } else {
                    uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + qh * VD + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[e] = make_uint4(pack(o[8 * e] * inv, o[8 * e + 1] * inv),
                                          pack(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                          pack(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                          pack(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
                }
            }
        }
    }
    __syncwarp();
    // neither CTA leaves while the other's products or signals still reach it
    tc_fence_before();
    cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

template <int VD>
cudaError_t launch(const ExpandedArgs& a, cudaStream_t st) {
    const uint64_t rows = (uint64_t)a.b.total_rows, heads = (uint64_t)a.heads;
    const uint64_t d = (uint64_t)(a.nope + a.rope);
    CUtensorMap tq, tk, tr, tv;
    auto heads_map = [&](CUtensorMap* m, const void* base, uint64_t width, uint64_t n, uint32_t box) {
        const uint64_t dims[3] = {width, heads, n}, strides[2] = {width * 2, heads * width * 2};
        const uint32_t b[3] = {64, 1, box};
        return encode_bf16_map(m, base, 3, dims, strides, b);
    };
    if (!heads_map(&tq, a.q, d, (uint64_t)a.b.n_q, kRows) ||
        !heads_map(&tk, a.k_nope, (uint64_t)a.nope, rows, kK / 2) || !heads_map(&tv, a.v, VD, rows, kK))
        return cudaErrorInvalidValue;
    tr = tk;
    if (a.rope > 0) {
        const uint64_t dims[2] = {(uint64_t)a.width, rows}, strides[1] = {(uint64_t)a.width * 2};
        const uint32_t b[2] = {64, kK / 2};
        if (!encode_bf16_map(&tr, a.rows, 2, dims, strides, b)) return cudaErrorInvalidValue;
    }
    auto kern = expanded_tc<VD>;
    cudaError_t e = ensure_dyn_smem((const void*)kern, (int)kSmem);
    if (e != cudaSuccess) return e;
    const int nk = (int)(d / 64);
    int ring = (int)((kSmem - 1024 - kBarBytes - nk * kQBlock) / unit_size(nk, VD));
    if (ring > kMaxRing) ring = kMaxRing;
    const int64_t slots = expanded_slots(a.b.n_q, a.b.n_seq, kQ);
    return launch_pdl(kern, dim3((unsigned)(2 * slots * a.heads * a.n_split)), dim3(kThreads), kSmem, st, tq, tk, tr,
                      tv, a, (int32_t)slots, (int32_t)ring);
}

}  // namespace

cudaError_t launch_expanded_tc(const ExpandedArgs& a, cudaStream_t st) {
    return a.v_dim == 256 ? launch<256>(a, st) : launch<128>(a, st);
}

}  // namespace dsa
