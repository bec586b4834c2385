// expanded_mla_tc.cu -- causal attention over expanded keys and values on the
// tcgen05 tensor cores (bf16).
//
//   S = Q K^T (M = 256 queries, N = 128 keys, K = the head's width), one pass over
//   the key tiles with a running maximum, O += P V (M = 256, N = v_dim, K = 128 keys)
//
// A unit of work is a tile of 256 queries of a sequence and a head; a pair of CTAs
// (cta_group::2) takes one after the other, each with 128 of the queries, their S, P and O, and
// half of the keys' rows and of the values' columns to load.
// The next unit is one whose launch the pair cancels (clusterlaunchcontrol), asked for a unit
// ahead, so that its copies and first products run while the last one's output is written.
// In each CTA
//   warp 8     TMA: the queries, and a ring of a tile's keys (columns in blocks of 64, the
//              rope block from the cache rows, for every head) or a tile's values in
//              the order of their use; hands out the units of work;
//   warp 9     in the first CTA issues the products for both, S of tile t + 1 before O
//              of tile t, from one unit of work into the next;
//   warps 0-7  softmax, a query row and half of its keys to a thread: S from TMEM,
//              exp, P in bf16 back over S (O takes it from TMEM as its A operand).
//              Row maxima are raised only when a logit exceeds them by more than
//              kSlack, so the two halves of a row share a maximum without telling each
//              other theirs: a barrier that also votes says whether any row is raised,
//              and only then they are exchanged and O is rescaled in TMEM;
//   warps 10-11 values of tiles that some query sees only in part: NaN and infinities
//              are taken out of shared memory (0 times either is NaN) and given back in the
//              epilogue to the queries that see them; and the check of the sequences' offsets;
//   warps 12-15 epilogue: a unit's O to the output beside the next unit's first scores, a
//              row to a thread, 64 columns of a warp's rows at a time through shared memory
//              and a TMA store; straight from registers in whole sectors where a
//              sequence ends among the warp's rows.  (From registers always: 64 prompts of 200
//              tokens 260 us instead of 242, the stores of 32 rows each keep the softmax
//              out of the load-store unit.)
// A key tile takes 2,050 cycles (head width and v_dim 256), which are the products' own: S
// and O of 1,024 each.  What it took before: a unit's launch to itself, with its start, its
// output and nothing beside them, 11,000 cycles; copies and products handed over in eight
// blocks a tile, 3,700 cycles a tile, some 200 a hand-over; arrivals that release to the
// cluster, 1,000 to 3,000 cycles each (sm100.cuh).
// P is rounded to bf16 because both operands of the value product have one
// type and V is bf16: 2^-8 of a weight at most, of random sign.
#include <math.h>

#include "expanded_mla.cuh"
#include "pair.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kQ = kExpandedTcQ, kK = kExpandedTcK;      // queries and keys of a tile
constexpr int kRows = kQ / 2;                            // queries of a CTA
constexpr uint32_t kQBlock = kRows * 128;                // 64 columns of them
constexpr uint32_t kKBlock = kK / 2 * 128;               // 64 columns of a CTA's half of a tile's keys
constexpr int kMaxRing = 11;
constexpr int kWorks = 4;                                // units of work handed out at a time
constexpr int kSoftmax = 256;                            // threads
constexpr int kTmaWarp = 8, kMmaWarp = 9, kCleanWarp = 10, kOutWarp = 12;
constexpr int kThreads = 512;                            // 128 registers each at the launch, then
// of the softmax's 256 threads and of the others
constexpr int kSoftmaxRegs = 144, kOtherRegs = 112;
constexpr int kCleaners = 64;
constexpr uint32_t kOCol = 256, kTmemCols = 512;         // S0, S1 at 0 and 128
constexpr uint32_t kSmem = 227 * 1024;
constexpr uint32_t kBarBytes = 5120;
constexpr uint32_t kStage = 32 * 128;                    // 64 columns of an epilogue warp's rows
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;                            // weights stay below 2^8

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A unit of work as the roles read it.
struct Work {
    int64_t q0, row0, first;                             // as ExpandedTile, of the pair
    int32_t n_q, n;                                      // n: its key tiles, -1: no more work
    int32_t partial;                                     // key tiles from this one on are not seen in full by every query
    int32_t h;
    uint32_t unit;                                       // its number: each is handed out once
};

struct Shared {
    uint64_t full[kMaxRing], empty[kMaxRing], part[kMaxRing], clean[kMaxRing];
    uint64_t q_full, q_free, s_full[2], p_full[2], o_done, o_free, o_last, drain;
    uint64_t l_full[2];
    uint64_t work_full[kWorks], work_free[kWorks], next_full[2], next_free[2];
    alignas(16) uint4 next[2];                           // answers to the requests for work
    Work work[kWorks];
    float l[2][kSoftmax], m[2][kRows];                   // a unit's sums of halves, and its maxima
    uint32_t tmem;
    int32_t abort;
    // the last unit that met odd values, by its number: the cleaners may be two units ahead of
    // the epilogue (their queries' place is free once a unit's scores are issued), not three
    int32_t poison[4];
};
static_assert(sizeof(Shared) <= kBarBytes, "barriers");

// Asks for a cluster that has not been launched, in its place; the answer goes to
// both CTAs of the pair.
__device__ __forceinline__ void ask_work(uint4* answer, uint64_t* bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(smem_u32(answer)), "r"(smem_u32(bar))
        : "memory");
}
// The first block of the cluster that the answer gives, or -1.
__device__ __forceinline__ int64_t answer_block(const uint4* answer) {
    uint32_t given, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
        : "=r"(given), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    return given ? (int64_t)x : -1;
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

// Room for either kind of unit.
__host__ __device__ constexpr uint32_t unit_size(int nk, int v_dim) {
    const uint32_t k = nk * kKBlock, v = v_dim / 128 * (kK * 128);
    return k > v ? k : v;
}

template <int VD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
expanded_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
            const __grid_constant__ CUtensorMap tm_o, const ExpandedArgs a, const int32_t slots, const int32_t ring) {
    constexpr uint32_t kVBlock = kK * 128;               // 64 columns of a tile's values
    constexpr uint32_t kVBytes = VD / 128 * kVBlock;     // a CTA's half of them
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Shared& s = *reinterpret_cast<Shared*>(smem);
    uint8_t* Qs = smem + kBarBytes;
    const int nk = (a.nope + a.rope) / 64, nope_blocks = a.nope / 64;   // blocks of a tile's keys
    const uint32_t unit_bytes = unit_size(nk, VD);       // of the ring
    uint8_t* Rs = Qs + nk * kQBlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxRing; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
            mbar_init(&s.part[i], 1);
            mbar_init(&s.clean[i], 2 * kCleaners / 32);
        }
        mbar_init(&s.q_full, 1);
        mbar_init(&s.q_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 2 * kSoftmax / 32);
            mbar_init(&s.next_full[i], 1);
            mbar_init(&s.next_free[i], 1);
        }
        for (int i = 0; i < 4; ++i) s.poison[i] = 0;
        for (int i = 0; i < kWorks; ++i) {
            mbar_init(&s.work_full[i], 1);
            // the softmax's, the cleaners' and the epilogue's warps, and the products' thread
            mbar_init(&s.work_free[i], (kSoftmax + kCleaners + kRows) / 32 + (rank == 0 ? 1 : 0));
        }
        mbar_init(&s.o_done, 1);
        mbar_init(&s.o_free, 2 * kRows / 32);
        for (int i = 0; i < 2; ++i) mbar_init(&s.l_full[i], kSoftmax / 32);
        mbar_init(&s.o_last, 1);
        mbar_init(&s.drain, 1);
        s.abort = 0;
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
    if (warp < kTmaWarp) regs_inc<kSoftmaxRegs>();
    else regs_dec<kOtherRegs>();

    if (warp == kTmaWarp) {
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
            int64_t block = blockIdx.x - rank;                     // the pair's
            int busy = 0;                                          // units of work with key tiles so far
            bool asked = false;
            for (uint32_t k = 0; ok; ++k) {
                // ask for the unit after this one: the request needs both CTAs' leave
                if (block >= 0) {
                    mbar_arrive_expect_tx(&s.next_full[k & 1], 16);
                    if (rank == 0) {
                        ok = k < 2 || wait(&s.next_free[k & 1], ((k >> 1) - 1) & 1, abort);
                        if (!ok) break;
                        ask_work(&s.next[k & 1], &s.next_full[k & 1]);
                    }
                    asked = true;
                }
                // this one: a head's tiles one after the other (its keys and values stay in
                // L2), the longest first
                ExpandedTile t;
                Work w;
                w.n = -1;
                if (block >= 0) {
                    w.unit = (uint32_t)(block / 2);
                    w.h = (int)(w.unit / slots);
                    const int64_t slot = slots - 1 - (int64_t)(w.unit % slots);
                    if (!expanded_tile(a.b, slot, 0, 1, kQ, kK, t)) {
                        t.n_q = t.kt1 = 0;
                        t.q0 = t.row0 = t.first = 0;
                    }
                    w.q0 = t.q0; w.row0 = t.row0; w.first = t.first;
                    w.n_q = t.n_q; w.n = t.kt1;
                    w.partial = (int)(t.first / kK);
                }
                ok = k < kWorks || wait(&s.work_free[k % kWorks], (k / kWorks - 1) & 1, abort);
                if (!ok) break;
                s.work[k % kWorks] = w;
                mbar_arrive(&s.work_full[k % kWorks]);
                if (w.n < 0) break;
                if (w.n > 0) {
                    auto keys = [&](int kt) {                      // half of the tile's rows
                        const int32_t y = (int32_t)(w.row0 + (int64_t)kt * kK + rank * (kK / 2));
                        uint32_t bar;
                        uint8_t* dst = next(nk * kKBlock, bar, false);
                        for (int b = 0; b < nk && ok; ++b) {
                            if (b < nope_blocks) tma_load_3d_pair(dst + b * kKBlock, &tm_k, bar, b * 64, w.h, y);
                            else tma_load_2d_pair(dst + b * kKBlock, &tm_r, bar, a.kv_lora + (b - nope_blocks) * 64, y);
                        }
                    };
                    auto values = [&](int kt) {                    // half of the columns
                        const int32_t y = (int32_t)(w.row0 + (int64_t)kt * kK);
                        uint32_t bar;
                        uint8_t* dst = next(kVBytes, bar, kt >= w.partial);
                        for (int c = 0; c < VD / 128 && ok; ++c)
                            tma_load_3d_pair(dst + c * kVBlock, &tm_v, bar, rank * (VD / 2) + c * 64, w.h, y);
                    };
                    ok = (busy == 0 || wait(&s.q_free, (busy - 1) & 1, abort));
                    if (!ok) break;
                    if (rank == 0) mbar_arrive_expect_tx(&s.q_full, 2 * nk * kQBlock);
                    for (int b = 0; b < nk; ++b)
                        tma_load_3d_pair(Qs + b * kQBlock, &tm_q, cluster_addr(&s.q_full, 0), b * 64, w.h,
                                         (int32_t)(w.q0 + rank * kRows));
                    keys(0);
                    for (int i = 0; i < w.n && ok; ++i) {
                        if (i + 1 < w.n) keys(i + 1);
                        if (ok) values(i);
                    }
                    ++busy;
                }
                ok = ok && wait(&s.next_full[k & 1], (k >> 1) & 1, abort);
                if (!ok) break;
                asked = false;
                block = answer_block(&s.next[k & 1]);
                fence_proxy_async_smem();                          // read before the next answer is written
                if (rank != 0) mbar_arrive_cluster(cluster_addr(&s.next_free[k & 1], 0));
            }
            if (!ok) {
                record_error(a.err, kDevTimeout, blockIdx.x, 62);
                *abort = 1;
                // copies and answers in flight land first: their barriers are partly the other CTA's
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < (asked ? 100000000ull : 50000000ull)) {}
            }
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0 && elect_one()) {                            // ---- products
            bool ok = true;
            Place p;
            uint32_t g = 0, busy = 0, k = 0;                       // key tiles, units with some, units so far
            uint32_t cleaned = 0;                                  // parities of the clean barriers
            const uint32_t q_addr = smem_u32(Qs), r_addr = smem_u32(Rs);
            const uint32_t id_s = idesc_bf16_f32(kQ, kK), id_o = idesc_bf16_f32_major(kQ, VD, 0, 1);
            auto scores = [&](uint32_t tile, const Place& at) {
                ok = ok && wait(&s.full[at.at], at.parity, abort);
                if (!ok) return;
                tc_fence_after();
                const uint32_t k_addr = r_addr + at.at * unit_bytes, d = tmem + (tile & 1) * kK;
                for (int b = 0; b < nk; ++b) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ss_pair(d, sdesc_kmajor_sw128(q_addr + b * kQBlock + kk * 32),
                                         sdesc_kmajor_sw128(k_addr + b * kKBlock + kk * 32), id_s, (b | kk) != 0);
                }
                mma_commit_pair(&s.empty[at.at]);
                mma_commit_pair(&s.s_full[tile & 1]);
            };
            auto values = [&](uint32_t tile, bool more, bool partly) {
                ok = ok && wait(&s.full[p.at], p.parity, abort);
                if (ok && partly) {
                    ok = wait(&s.clean[p.at], (cleaned >> p.at) & 1, abort);
                    cleaned ^= 1u << p.at;
                }
                ok = ok && wait(&s.p_full[tile & 1], (tile >> 1) & 1, abort);
                if (!ok) return;
                tc_fence_after();
                const uint32_t v_addr = r_addr + p.at * unit_bytes, w = tmem + (tile & 1) * kK;
#pragma unroll
                for (int kk = 0; kk < kK / 16; ++kk)
                    mma_bf16_ts_pair(tmem + kOCol, w + kk * 8, sdesc_sw128(v_addr + kk * 2048, kVBlock, 1024), id_o,
                                     more || kk != 0);
                mma_commit_pair(&s.empty[p.at]);
                mma_commit_pair(&s.o_done);
            };
            // the next unit with key tiles: known (1), not yet handed out (0), none (-1)
            int known = 0, n_next = 0, partial_next = 0;
            auto fetch = [&](bool blocking) {
                while (known == 0) {
                    uint64_t* bar = &s.work_full[k % kWorks];
                    const uint32_t parity = (k / kWorks) & 1;
                    if (!blocking && !mbar_test_wait(bar, parity)) return;
                    ok = ok && wait(bar, parity, abort);
                    if (!ok) return;
                    n_next = s.work[k % kWorks].n;
                    partial_next = s.work[k % kWorks].partial;
                    mbar_arrive(&s.work_free[k % kWorks]);
                    ++k;
                    known = n_next < 0 ? -1 : n_next > 0 ? 1 : 0;
                }
            };
            bool early = false;                                    // the unit's first scores are issued
            fetch(true);
            while (ok && known == 1) {
                const int n = n_next, partial = partial_next;
                known = 0;
                if (!early) {
                    ok = wait(&s.q_full, busy & 1, abort);
                    scores(g, p);
                    p.step(ring);
                }
                early = false;
                for (int i = 0; i < n && ok; ++i) {
                    if (i + 1 < n) {
                        scores(g + i + 1, p);
                        p.step(ring);
                    }
                    if (i == (n > 1 ? n - 2 : 0)) mma_commit_pair(&s.q_free);   // the last scores are issued
                    // the last unit's O has been read
                    if (i == 0 && busy > 0) ok = ok && wait(&s.o_free, (busy - 1) & 1, abort);
                    if (i == n - 1) {
                        // the next unit's first scores, if they can begin before these weights
                        // are there; its keys lie behind this tile's values in the ring
                        Place after = p;
                        after.step(ring);
                        const long long t0 = clock64();
                        while (ok && !mbar_test_wait(&s.p_full[(g + i) & 1], ((g + i) >> 1) & 1)) {
                            if (known == 0) fetch(false);
                            if (known == 1 && mbar_test_wait(&s.q_full, (busy + 1) & 1) &&
                                mbar_test_wait(&s.full[after.at], after.parity)) {
                                scores(g + n, after);
                                early = true;
                                break;
                            }
                            if (*abort != 0 || clock64() - t0 > kWaitCycles) ok = false;
                        }
                    }
                    values(g + i, i > 0, i >= partial);
                    p.step(ring);
                    if (early) p.step(ring);
                }
                if (ok) mma_commit_pair(&s.o_last);
                g += n;
                ++busy;
                if (ok) fetch(true);
            }
            if (!ok) {
                record_error(a.err, kDevTimeout, blockIdx.x, 63);
                *abort = 1;
                mma_commit_pair(&s.drain);                         // every issued product retired
                mbar_wait(&s.drain, 0, 50000000ull);
            }
        }
        __syncwarp();
    } else if (warp >= kCleanWarp && warp < kOutWarp) {            // ---- hidden values
        const int c = threadIdx.x - kCleanWarp * 32;
        uint32_t parted = 0;                                       // parities of the part barriers
        uint32_t before = 0;                                       // units of the ring before this work's
        int32_t busy = 0;
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            ok = warp_wait(&s.work_full[k % kWorks], (k / kWorks) & 1, abort);
            if (!ok) break;
            const int n = s.work[k % kWorks].n;
            const int partial = s.work[k % kWorks].partial;
            const uint32_t unit = s.work[k % kWorks].unit;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.work_free[k % kWorks]);
            if (n < 0) break;
            // the pair's share of the sequences, in warps that mostly have nothing to do
            expanded_check(a.b, ((int64_t)unit * 2 + rank) * kCleaners + c, (int64_t)slots * a.heads * 2 * kCleaners, a.err,
                           61);
            if (n == 0) continue;
            ++busy;
            for (int i = partial; i < n; ++i) {
                // before tile i's values: keys of tiles 0 .. min(i + 1, n - 1), values of 0 .. i - 1
                const uint32_t at = (before + (uint32_t)((i + 1 < n ? i + 2 : n) + i)) % ring;
                ok = warp_wait(&s.part[at], (parted >> at) & 1, abort);
                parted ^= 1u << at;
                if (!ok) break;
                uint4* p = reinterpret_cast<uint4*>(Rs + at * unit_bytes) + c;
                // an exponent of ones carries into its half's sign
                auto odd = [](uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                bool bad = false;
#pragma unroll 1
                for (int e0 = 0; e0 < (int)(kVBytes / 16 / kCleaners); e0 += 8) {
                    uint4 x[8];
                    uint32_t any = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = p[(e0 + e) * kCleaners];
#pragma unroll
                    for (int e = 0; e < 8; ++e) any |= odd(x[e].x) | odd(x[e].y) | odd(x[e].z) | odd(x[e].w);
                    if (any == 0) continue;
                    bad = true;
                    // the halves that are odd become zeros
                    auto clean = [&](uint32_t w) { return w & ~((odd(w) >> 15) * 0xffffu); };
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        p[(e0 + e) * kCleaners] = make_uint4(clean(x[e].x), clean(x[e].y), clean(x[e].z), clean(x[e].w));
                }
                if (bad) {                                         // both CTAs give them back
                    *(volatile int32_t*)&s.poison[busy & 3] = busy;
                    st_cluster(cluster_addr(&s.poison[busy & 3], rank ^ 1), busy);
                    fence_cluster();
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(&s.clean[at], 0));
            }
            before = (before + 2u * (uint32_t)n) % ring;
        }
        if (!ok) {
            if (lane == 0) record_error(a.err, kDevTimeout, blockIdx.x, 64);
            *abort = 1;
        }
    } else if (warp < kTmaWarp) {                                  // ---- softmax
        const int row = (int)rank * kRows + (threadIdx.x & 127);   // of the pair's queries
        const int half = threadIdx.x >> 7;
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float scale = a.scale * kLog2e;
        uint32_t g = 0, busy = 0;
        bool ok = true;
        for (uint32_t k = 0; ; ++k) {
            ok = ok && warp_wait(&s.work_full[k % kWorks], (k / kWorks) & 1, abort);
            if (softmax_vote(!ok)) { ok = false; break; }          // all go on, or none
            const Work& w = s.work[k % kWorks];
            const int n = w.n, partial = w.partial;
            const int64_t sees = w.first + row;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.work_free[k % kWorks]);
            if (n < 0) break;
            if (n == 0) continue;
            float m = -INFINITY, l = 0.f;                          // l: of this half's keys
            for (int i = 0; i < n; ++i, ++g) {
                // a warp that gives up votes and meets the others all the same
                ok = ok && warp_wait(&s.s_full[g & 1], (g >> 1) & 1, abort);
                tc_fence_after();
                const uint32_t at = lane_addr + (g & 1) * kK;
                float v[2][32];
                tmem_ld_32cols_x2(at + half * 64, at + half * 64 + 32, v[0], v[1]);
                if (i >= partial) {
                    // this half's keys of the tile that the row sees
                    const int64_t here = sees - (int64_t)i * kK - half * 64;
                    const int left = here < 0 ? 0 : here > 64 ? 64 : (int)here;
                    if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (e >= left) v[e >> 5][e & 31] = -INFINITY;
                    }
                }
                float tops[4] = {v[0][0], v[0][1], v[0][2], v[0][3]};
#pragma unroll
                for (int e = 4; e < 64; ++e) tops[e & 3] = fmaxf(tops[e & 3], v[e >> 5][e & 31]);
                float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale;
                // of -inf: any logit above it
                if (softmax_vote(top > m + kSlack || !ok)) {
                    // through the columns of S behind P: the products leave shared memory
                    // little bandwidth for others
                    tmem_st_1col(at + kK / 2 + half, top);
                    tc_fence_before();
                    ok = !softmax_vote(!ok);
                    if (!ok) break;
                    tc_fence_after();
                    top = fmaxf(top, tmem_ld_1col(at + kK / 2 + (half ^ 1)));
                    const float mn = top > m + kSlack ? top : m;
                    const float f = mn == m ? 1.f : ex2(m - mn);
                    if (__any_sync(0xffffffffu, mn != m) && i > 0) {
                        ok = warp_wait(&s.o_done, (g - 1) & 1, abort);
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
                }
                const float base = m == -INFINITY ? 0.f : -m;      // no logit above -inf yet
                const float2 scale2 = make_float2(scale, scale), base2 = make_float2(base, base);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                float x[32];
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    float2 p = fma_x2(make_float2(v[e >> 5][e & 31], v[e >> 5][(e & 31) + 1]), scale2, base2);
                    p.x = ex2(p.x);
                    p.y = ex2(p.y);
                    sum[(e >> 1) & 1] = add_x2(sum[(e >> 1) & 1], p);
                    x[e >> 1] = __uint_as_float(pack(p.x, p.y));
                }
                tmem_st_32cols(at + half * 32, x);
                const float2 both = add_x2(sum[0], sum[1]);
                l += both.x + both.y;
                tc_fence_before();
                __syncwarp();
                if (ok && lane == 0) mbar_arrive_cluster(cluster_addr(&s.p_full[g & 1], 0));
            }
            // for the epilogue, which has read those of the unit before the last: that O is free
            s.l[busy & 1][threadIdx.x] = l;
            if (half == 0) s.m[busy & 1][threadIdx.x] = m;
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&s.l_full[busy & 1]);
            ++busy;
        }
        if (!ok) {
            if (lane == 0) record_error(a.err, kDevTimeout, blockIdx.x, 65);
            *abort = 1;
        }
    } else {                                                       // ---- epilogue
        const int r = threadIdx.x & 127, row = (int)rank * kRows + r;
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        uint8_t* stage = Rs + ring * unit_bytes + (warp & 3) * kStage;
        int32_t busy = 0;
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            ok = warp_wait(&s.work_full[k % kWorks], (k / kWorks) & 1, abort);
            if (!ok) break;
            const Work w = s.work[k % kWorks];
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.work_free[k % kWorks]);
            if (w.n < 0) break;
            const int64_t qh = (w.q0 + row) * a.heads + w.h;
            const bool mine = row < w.n_q;
            if (w.n == 0) continue;
            // the softmax may be two units ahead of this, hence its two barriers
            ok = warp_wait(&s.l_full[busy & 1], (busy >> 1) & 1, abort) && warp_wait(&s.o_last, busy & 1, abort);
            if (!ok) break;
            tc_fence_after();
            const float l = s.l[busy & 1][r] + s.l[busy & 1][r + 128], m = s.m[busy & 1][r];
            ++busy;
            const bool poison = *(volatile int32_t*)&s.poison[busy & 3] == busy;
            if (poison) {                                          // what the cleaners took out and the row sees
                const int64_t from = (int64_t)w.partial * kK, to = mine ? w.first + row : from;
#pragma unroll 1
                for (int c = 0; c < VD; c += 32) {
                    float o[32];
                    tmem_ld_32cols(lane_addr + kOCol + c, o);
#pragma unroll 1
                    for (int64_t j = from; j < to; ++j) {
                        const __nv_bfloat16* y = static_cast<const __nv_bfloat16*>(a.v) +
                                                 ((w.row0 + j) * a.heads + w.h) * VD + c;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float z = __bfloat162float(y[e]);
                            if (!isfinite(z)) o[e] += z;
                        }
                    }
                    __syncwarp();
                    tmem_st_32cols(lane_addr + kOCol + c, o);
                }
            }
            const float inv = 1.f / l;
            const int r0 = (int)rank * kRows + (warp & 3) * 32;    // the warp's first query
            const bool whole = r0 + 32 <= w.n_q;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + qh * VD;
#pragma unroll 1
            for (int c = 0; c < VD; c += 64) {
                uint32_t x[32];
                {
                    float o[2][32];
                    tmem_ld_32cols_x2(lane_addr + kOCol + c, lane_addr + kOCol + c + 32, o[0], o[1]);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        x[e] = pack(o[e >> 4][(e & 15) * 2] * inv, o[e >> 4][(e & 15) * 2 + 1] * inv);
                }
                if (c + 64 == VD) {                                // O may be written again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(cluster_addr(&s.o_free, 0));
                }
                if (whole) {
                    if (lane == 0) tma_store_wait_read<0>();       // the piece before has left
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e)                    // the map's 128-byte swizzle
                        *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                            make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&tm_o, stage, c, w.h, (int32_t)(w.q0 + r0));
                        tma_store_commit();
                    }
                } else if (mine) {                                 // the rows behind are another sequence's
#pragma unroll
                    for (int e = 0; e < 4; ++e) store_sector(out + c + e * 16, &x[8 * e]);
                }
            }
            if (mine && a.lse != nullptr) a.lse[qh] = expanded_lse(m, l);
        }
        if (lane == 0) tma_store_wait<0>();
        if (!ok) {
            if (lane == 0) record_error(a.err, kDevTimeout, blockIdx.x, 66);
            *abort = 1;
        }
    }
    // neither CTA leaves while the other's products or signals still reach it
    __syncwarp();
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
    CUtensorMap tq, tk, tr, tv, to;
    auto heads_map = [&](CUtensorMap* m, const void* base, uint64_t width, uint64_t n, uint32_t box) {
        const uint64_t dims[3] = {width, heads, n}, strides[2] = {width * 2, heads * width * 2};
        const uint32_t b[3] = {64, 1, box};
        return encode_bf16_map(m, base, 3, dims, strides, b);
    };
    if (!heads_map(&tq, a.q, d, (uint64_t)a.b.n_q, kRows) ||
        !heads_map(&tk, a.k_nope, (uint64_t)a.nope, rows, kK / 2) || !heads_map(&tv, a.v, VD, rows, kK) ||
        !heads_map(&to, a.out, VD, (uint64_t)a.b.n_q, 32))
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
    int ring = (int)((kSmem - 1024 - kBarBytes - nk * kQBlock - 4 * kStage) / unit_size(nk, VD));
    if (ring > kMaxRing) ring = kMaxRing;
    const int64_t slots = expanded_slots(a.b.n_q, a.b.n_seq, kQ);
    return launch_pdl(kern, dim3((unsigned)(2 * slots * a.heads)), dim3(kThreads), kSmem, st, tq, tk, tr,
                      tv, to, a, (int32_t)slots, (int32_t)ring);
}

}  // namespace

cudaError_t launch_expanded_tc(const ExpandedArgs& a, cudaStream_t st) {
    return a.v_dim == 256 ? launch<256>(a, st) : launch<128>(a, st);
}

}  // namespace dsa
