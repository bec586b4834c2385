// expanded_mla_tc.cu -- causal attention over expanded keys and values on the
// tcgen05 tensor cores (bf16).
//
//   S = Q K^T (M = 128 queries, N = 128 keys, K = the head's width), one pass over
//   the key tiles with a running maximum, O += P V (M = 128, N = v_dim, K = 128 keys)
//
// One CTA per (tile of 128 queries, head, split of the key tiles):
//   warp 8     TMA: the queries once, then a ring of 16 KB blocks in the order of
//              their use -- a tile's keys as blocks of 64 columns (the rope block from
//              the cache rows, for every head), its values as blocks of 8192 / v_dim keys;
//   warp 9     issues the products, S of tile t + 1 before O of tile t;
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
constexpr uint32_t kBlock = 16384;
constexpr int kMaxRing = 13;
constexpr int kSoftmax = 256;                            // threads
constexpr int kTmaWarp = 8, kMmaWarp = 9, kCleanWarp = 10;
constexpr int kThreads = 384;
constexpr int kCleaners = 64;
constexpr uint32_t kOCol = 256, kTmemCols = 512;         // S0, S1 at 0 and 128
constexpr uint32_t kSmem = 227 * 1024;
constexpr uint32_t kBarBytes = 2048;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;                            // weights stay below 2^8

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D[tmem] (+)= A[tmem] * B[smem], bf16.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b),
        "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

struct Bars {
    uint64_t full[kMaxRing], empty[kMaxRing], turn[kMaxRing], clean[kMaxRing];
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

// A wait that a whole warp makes: all lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort) {
    const bool ok = *abort == 0 && mbar_wait(bar, parity, kWaitNs);
    return __all_sync(0xffffffffu, ok);
}

template <int VD>
__global__ void __launch_bounds__(kThreads, 1)
expanded_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
            const ExpandedArgs a, const int32_t slots, const int32_t ring) {
    constexpr int kKeysV = 8192 / VD;                    // keys of a block of values
    constexpr int kBlocksV = kK / kKeysV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Bars& s = *reinterpret_cast<Bars*>(smem);
    uint8_t* Qs = smem + kBarBytes;
    const int nk = (a.nope + a.rope) / 64, nope_blocks = a.nope / 64;   // blocks of a tile's keys
    uint8_t* Rs = Qs + nk * kBlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a head's tiles one after the other (its keys and values stay in L2), the
    // longest first
    const int split = (int)(blockIdx.x % a.n_split);
    const int64_t slot = slots - 1 - (int64_t)(blockIdx.x / a.n_split) % slots;
    const int h = (int)(blockIdx.x / a.n_split / slots);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxRing; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
            mbar_init(&s.turn[i], 1);
            mbar_init(&s.clean[i], kCleaners);
        }
        mbar_init(&s.q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], kSoftmax / 32);
        }
        mbar_init(&s.o_done, 1);
        mbar_init(&s.o_last, 1);
        mbar_init(&s.drain, 1);
        s.abort = 0;
        s.poison = 0;
        fence_mbarrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s.tmem, kTmemCols);
        tmem_relinquish();
    }
    if (warp == kTmaWarp && lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_r);
        prefetch_tensormap(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
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
            int used = 0;                                          // blocks so far
            Place p;
            auto next = [&](uint8_t*& dst, uint64_t*& bar, bool partly = false) {
                ok = *abort == 0 && mbar_wait(&s.empty[p.at], p.parity ^ 1, kWaitNs);
                if (!ok) return false;
                dst = Rs + p.at * kBlock;
                bar = &s.full[p.at];
                mbar_arrive_expect_tx(bar, kBlock);
                // the cleaners' turn: they do not follow the ring, so its barrier's
                // phase alone would not tell them this use from an earlier one
                if (partly) mbar_arrive(&s.turn[p.at]);
                ++used;
                p.step(ring);
                return true;
            };
            auto keys = [&](int kt) {
                const int32_t y = (int32_t)(t.row0 + (int64_t)kt * kK);
                for (int b = 0; b < nk; ++b) {
                    uint8_t* dst;
                    uint64_t* bar;
                    if (!next(dst, bar)) return;
                    if (b < nope_blocks) tma_load_3d(dst, &tm_k, bar, b * 64, h, y);
                    else tma_load_2d(dst, &tm_r, bar, a.kv_lora + (b - nope_blocks) * 64, y);
                }
            };
            auto values = [&](int kt) {
                const int32_t y = (int32_t)(t.row0 + (int64_t)kt * kK);
                for (int b = 0; b < kBlocksV; ++b) {
                    uint8_t* dst;
                    uint64_t* bar;
                    if (!next(dst, bar, kt >= partial)) return;
                    for (int c = 0; c < VD / 64; ++c)
                        tma_load_3d(dst + c * (kKeysV * 128), &tm_v, bar, c * 64, h, y + b * kKeysV);
                }
            };
            mbar_arrive_expect_tx(&s.q_full, nk * kBlock);
            for (int b = 0; b < nk; ++b) tma_load_3d(Qs + b * kBlock, &tm_q, &s.q_full, b * 64, h, (int32_t)t.q0);
            keys(t.kt0);
            for (int i = 0; i < n && ok; ++i) {
                if (i + 1 < n) keys(t.kt0 + i + 1);
                if (ok) values(t.kt0 + i);
            }
            if (!ok) {
                record_error(a.err, kDevTimeout, blockIdx.x, 62);
                *abort = 1;
                // copies in flight land first
                mbar_wait(&s.q_full, 0, 50000000ull);
                for (int u = used > ring ? used - ring : 0; u < used; ++u)
                    mbar_wait(&s.full[u % ring], (u / ring) & 1, 50000000ull);
            }
        }
    } else if (n > 0 && warp == kMmaWarp) {
        if (elect_one()) {                                         // ---- products
            bool ok = mbar_wait(&s.q_full, 0, kWaitNs);
            Place p;
            uint32_t cleaned = 0;                                  // parities of the clean barriers
            const uint32_t q_addr = smem_u32(Qs), r_addr = smem_u32(Rs);
            const uint32_t id_s = idesc_bf16_f32(kQ, kK), id_o = idesc_bf16_f32_major(kQ, VD, 0, 1);
            auto scores = [&](int i) {
                for (int b = 0; b < nk; ++b, p.step(ring)) {
                    const int at = p.at;
                    ok = ok && *abort == 0 && mbar_wait(&s.full[at], p.parity, kWaitNs);
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ss(tmem + (i & 1) * kK, sdesc_kmajor_sw128(q_addr + b * kBlock + kk * 32),
                                    sdesc_kmajor_sw128(r_addr + at * kBlock + kk * 32), id_s, (b | kk) != 0);
                    mma_commit(&s.empty[at]);
                }
                mma_commit(&s.s_full[i & 1]);
            };
            auto values = [&](int i) {
                ok = *abort == 0 && mbar_wait(&s.p_full[i & 1], (i >> 1) & 1, kWaitNs);
                for (int b = 0; b < kBlocksV; ++b, p.step(ring)) {
                    const int at = p.at;
                    ok = ok && *abort == 0 && mbar_wait(&s.full[at], p.parity, kWaitNs);
                    if (ok && t.kt0 + i >= partial) {
                        ok = mbar_wait(&s.clean[at], (cleaned >> at) & 1, kWaitNs);
                        cleaned ^= 1u << at;
                    }
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kKeysV / 16; ++kk)
                        mma_bf16_ts(tmem + kOCol, tmem + (i & 1) * kK + (b * kKeysV + kk * 16) / 2,
                                    sdesc_sw128(r_addr + at * kBlock + kk * 2048, kKeysV * 128, 1024), id_o,
                                    (i | b | kk) != 0);
                    mma_commit(&s.empty[at]);
                }
                mma_commit(&s.o_done);
            };
            scores(0);
            for (int i = 0; i < n && ok; ++i) {
                if (i + 1 < n) scores(i + 1);
                if (ok) values(i);
            }
            if (ok) {
                mma_commit(&s.o_last);
            } else {
                record_error(a.err, kDevTimeout, blockIdx.x, 63);
                *abort = 1;
                mma_commit(&s.drain);                              // every issued product retired
                mbar_wait(&s.drain, 0, 50000000ull);
            }
        }
        __syncwarp();
    } else if (n > 0 && warp >= kCleanWarp) {                               // ---- hidden values
        const int c = threadIdx.x - kCleanWarp * 32;
        uint32_t turned = 0;                                       // parities of the turn barriers
        for (int i = partial > t.kt0 ? partial - t.kt0 : 0; i < n; ++i) {
            // blocks used before tile i's values: keys of tiles 0 .. min(i + 1, n - 1), values of 0 .. i - 1
            const uint32_t first = (uint32_t)((i + 1 < n ? i + 2 : n) * nk + i * kBlocksV);
            bool ok = true;
            for (int b = 0; b < kBlocksV; ++b) {
                const uint32_t u = first + b, at = u % ring;
                ok = warp_wait(&s.turn[at], (turned >> at) & 1, abort) &&
                     warp_wait(&s.full[at], (u / ring) & 1, abort);
                turned ^= 1u << at;
                if (!ok) break;
                uint4* p = reinterpret_cast<uint4*>(Rs + at * kBlock);
                bool bad = false;
#pragma unroll 8
                for (int k = 0; k < (int)kBlock / 16 / kCleaners; ++k) {
                    uint4 x = p[c + k * kCleaners];
                    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
                    bool here = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if ((w[e] & 0x7f80u) == 0x7f80u) { w[e] &= 0xffff0000u; here = true; }
                        if ((w[e] & 0x7f800000u) == 0x7f800000u) { w[e] &= 0xffffu; here = true; }
                    }
                    if (here) { p[c + k * kCleaners] = x; bad = true; }
                }
                if (bad) *(volatile int32_t*)&s.poison = 1;
                fence_proxy_async_smem();
                mbar_arrive(&s.clean[at]);
            }
            if (!ok) {
                if (lane == 0) record_error(a.err, kDevTimeout, blockIdx.x, 64);
                *abort = 1;
                break;
            }
        }
    } else if (warp < kSoftmax / 32 && live) {                     // ---- softmax
        const int row = threadIdx.x & 127, half = threadIdx.x >> 7;
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
            if (ok && lane == 0) mbar_arrive(&s.p_full[i & 1]);
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
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
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
    if (!heads_map(&tq, a.q, d, (uint64_t)a.b.n_q, kQ) || !heads_map(&tk, a.k_nope, (uint64_t)a.nope, rows, kK) ||
        !heads_map(&tv, a.v, VD, rows, 8192 / VD))
        return cudaErrorInvalidValue;
    tr = tk;
    if (a.rope > 0) {
        const uint64_t dims[2] = {(uint64_t)a.width, rows}, strides[1] = {(uint64_t)a.width * 2};
        const uint32_t b[2] = {64, kK};
        if (!encode_bf16_map(&tr, a.rows, 2, dims, strides, b)) return cudaErrorInvalidValue;
    }
    auto kern = expanded_tc<VD>;
    cudaError_t e = ensure_dyn_smem((const void*)kern, (int)kSmem);
    if (e != cudaSuccess) return e;
    int ring = (int)((kSmem - 1024 - kBarBytes) / kBlock - d / 64);
    if (ring > kMaxRing) ring = kMaxRing;
    const int64_t slots = expanded_slots(a.b.n_q, a.b.n_seq, kQ);
    return launch_pdl(kern, dim3((unsigned)(slots * a.heads * a.n_split)), dim3(kThreads), kSmem, st, tq, tk, tr, tv,
                      a, (int32_t)slots, (int32_t)ring);
}

}  // namespace

cudaError_t launch_expanded_tc(const ExpandedArgs& a, cudaStream_t st) {
    return a.v_dim == 256 ? launch<256>(a, st) : launch<128>(a, st);
}

}  // namespace dsa
