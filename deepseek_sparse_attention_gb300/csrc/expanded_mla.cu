// expanded_mla.cu -- causal attention over expanded keys and values: float32 on
// CUDA cores, with the plan of its splits and their merge.  bf16 runs on the
// tensor cores (expanded_mla_tc.cu), without splits: 64 heads are 64 units of work
// for 76 pairs of CTAs, and seven splits of each were 2% faster over 130,000 rows,
// 10% slower over 30,000.
//
//   z_j = scale * (q_nope . k_nope[j, h] + q_rope . rope[j]),  j < L
//   out = sum_j softmax(z)_j v[j, h],  lse = log sum_j exp(z_j)
//
// The rope part of the key is the cache row's tail, shared by all heads.
//
// One CTA per (tile of 8 RPW queries, head, split of the key tiles): one pass over
// tiles of 32 keys with a running maximum and sum.  A warp has RPW queries.  Of
// their logits a lane sums a quarter of the columns (every fourth group of four) for
// all of them and four keys, so that an element read serves four or RPW products, and the
// quarters meet in shuffles that leave each lane its key.  Of the output a lane has every
// 32nd group of four columns.  Reads of shared memory and float32 arithmetic bound it
// about equally: 7,200 wavefronts and 8,200 cycles a tile of 64 queries.  (With a key
// to a lane, or two and 16 lanes to a query, 14,000 wavefronts.)
#include "expanded_mla.cuh"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kKeys = 32;
constexpr int kMaxTileQ = 64;                            // queries of the largest tile
constexpr int kMaxSplit = 16;
constexpr int64_t kSplitWaves = 2;                       // waves of a split call's CTAs, two to a multiprocessor
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// Shared memory: the queries, a tile of keys (rows padded by four against bank
// conflicts) and then its values in their place, the weights by key.  106 KB at
// the widest, so that two CTAs on a multiprocessor hide each other's loads.
__host__ __device__ constexpr int simt_smem_floats(int rows, int d, int v) {
    return rows * (d + 4) + kKeys * (d + 4 > v ? d + 4 : v) + kKeys * (rows + 4);
}

// A tile of up to 8 RPW queries.
template <int RPW, int VD>
__device__ __forceinline__ void simt_tile(const ExpandedArgs& a, const ExpandedTile& t, int h, int split, float* smem) {
    constexpr int BQ = 8 * RPW, kLdP = BQ + 4;
    constexpr int kVec = VD / 128;                       // groups of four output columns of a lane
    // Few queries, bound by the loads: these are asked for a product ahead, and warps without
    // a query do nothing else.  16 of them over up to 2,000 rows take 447 us, 4.1 TB/s; loads
    // where they are used, and two queries to every warp, 968.  (Tiles of 32 gain nothing from
    // loads ahead, tiles of 64 have no registers for them: 183 us instead of 174.)
    constexpr bool kAhead = RPW <= 2;
    const int d = a.nope + a.rope, ld = d + 4;
    float* Qs = smem;
    float* Ks = Qs + BQ * ld;
    float* Vs = Ks;
    float* Ps = Ks + kKeys * (ld > VD ? ld : VD);        // [key][query], rows of kLdP

    const float* q = static_cast<const float*>(a.q);
    const float* kn = static_cast<const float*>(a.k_nope);
    const float* rows = static_cast<const float*>(a.rows);
    const float* v = static_cast<const float*>(a.v);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;   // a warp's queries: warp + 8 r
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    // a warp copies every eighth row; its loads are all in flight before the first store
    // (one after the other they were 14,000 cycles a tile)
    for (int r0 = warp; r0 < BQ; r0 += 32) {
        float4 x[4][2];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = r0 + 8 * u, c = e * 128 + lane * 4;
                x[u][e] = r < t.n_q && c < d ? load4(q + ((t.q0 + r) * a.heads + h) * d + c) : zero;
            }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (r0 + 8 * u < BQ && e * 128 + lane * 4 < d) store4(Qs + (r0 + 8 * u) * ld + e * 128 + lane * 4, x[u][e]);
    }
    const bool busy = !kAhead || warp < t.n_q;
    float2 o[RPW][kVec][2] = {};
    float m[RPW], l[RPW];                                // l: of this lane's keys
#pragma unroll
    for (int r = 0; r < RPW; ++r) { m[r] = -INFINITY; l[r] = 0.f; }
    const float scale = a.scale * kLog2e;
    const int64_t last = t.first + t.n_q - 1;            // rows that the tile's last query sees
    // this warp's rows of a tile's keys, or of its values
    float4 x[4][2];
    auto load_keys = [&](int64_t j0) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = warp + 8 * u, c = e * 128 + lane * 4;
                const int64_t row = t.row0 + j0 + j;
                x[u][e] = j0 + j >= last || c >= d ? zero
                          : c < a.nope             ? load4(kn + (row * a.heads + h) * a.nope + c)
                                                   : load4(rows + row * a.width + a.kv_lora + c - a.nope);
            }
    };
    auto load_values = [&](int64_t j0) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const int64_t j = j0 + warp + 8 * u;
                x[u][e] = j < last ? load4(v + ((t.row0 + j) * a.heads + h) * VD + e * 128 + lane * 4) : zero;
            }
    };
    if (kAhead) load_keys((int64_t)t.kt0 * kKeys);

    for (int kt = t.kt0; kt < t.kt1; ++kt) {
        const int64_t j0 = (int64_t)kt * kKeys;
        if (!kAhead) load_keys(j0);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (e * 128 + lane * 4 < d) store4(Ks + (warp + 8 * u) * ld + e * 128 + lane * 4, x[u][e]);
        __syncthreads();
        if (kAhead) load_values(j0);
        if (busy) {
            const int quarter = lane >> 3, k8 = lane & 7;
            float s[RPW][4] = {};                        // of keys k8 + 8 k
#pragma unroll 1
            for (int c = quarter * 4; c < d; c += 16) {
                float4 k[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) k[e] = load4(Ks + (k8 + 8 * e) * ld + c);
#pragma unroll
                for (int r = 0; r < RPW; ++r) {
                    const float4 x = load4(Qs + (warp + 8 * r) * ld + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[r][e] = fmaf(x.x, k[e].x, fmaf(x.y, k[e].y, fmaf(x.z, k[e].z, fmaf(x.w, k[e].w, s[r][e]))));
                }
            }
            // the quarters' sums: a lane gives away those of the keys that it does not keep,
            // and keeps key k8 + 8 quarter = lane
            float p[RPW];
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                const bool hi = (quarter & 2) != 0, odd = (quarter & 1) != 0;
                const float a0 = (hi ? s[r][2] : s[r][0]) + __shfl_xor_sync(0xffffffffu, hi ? s[r][0] : s[r][2], 16);
                const float a1 = (hi ? s[r][3] : s[r][1]) + __shfl_xor_sync(0xffffffffu, hi ? s[r][1] : s[r][3], 16);
                const float dot = (odd ? a1 : a0) + __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 8);
                const float z = j0 + lane < t.first + warp + 8 * r ? dot * scale : -INFINITY;
                float top = z;
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float mn = fmaxf(m[r], top);
                const float base = mn == -INFINITY ? 0.f : mn;   // nothing to see so far
                const float f = exp2f(m[r] - base);
                p[r] = exp2f(z - base);
                l[r] = l[r] * f + p[r];
                m[r] = mn;
                const float2 f2 = make_float2(f, f);
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    o[r][c][0] = mul_x2(o[r][c][0], f2);
                    o[r][c][1] = mul_x2(o[r][c][1], f2);
                }
            }
            if constexpr (RPW == 8) {
                store4(Ps + lane * kLdP + warp * RPW, make_float4(p[0], p[1], p[2], p[3]));
                store4(Ps + lane * kLdP + warp * RPW + 4, make_float4(p[4], p[5], p[6], p[7]));
            } else {
#pragma unroll
                for (int r = 0; r < RPW; ++r) Ps[lane * kLdP + warp * RPW + r] = p[r];
            }
        }
        if (!kAhead) load_values(j0);
        __syncthreads();                                 // the keys are read, the warp's weights written
        float4 odd = zero;                               // NaN if a value is no number
        {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float4 y = x[u][e];
                    store4(Vs + (warp + 8 * u) * VD + e * 128 + lane * 4, y);
                    odd.x = fmaf(y.x, 0.f, odd.x); odd.y = fmaf(y.y, 0.f, odd.y);
                    odd.z = fmaf(y.z, 0.f, odd.z); odd.w = fmaf(y.w, 0.f, odd.w);
                }
        }
        if (kAhead && kt + 1 < t.kt1) load_keys(j0 + kKeys);
        // 0 times infinity is NaN: where some query does not see a key of the tile and a
        // value is no number, each weight is looked at
        const bool careful = __syncthreads_or((odd.x + odd.y) + (odd.z + odd.w) != 0.f) && j0 + kKeys > t.first;
        auto values = [&](int j, bool checked) {
            float w[RPW];
            if constexpr (RPW == 8) {
                const float4 x = load4(Ps + j * kLdP + warp * RPW), y = load4(Ps + j * kLdP + warp * RPW + 4);
                w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
            } else {
#pragma unroll
                for (int r = 0; r < RPW; ++r) w[r] = Ps[j * kLdP + warp * RPW + r];
            }
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                const float4 x = load4(Vs + j * VD + (c * 32 + lane) * 4);
#pragma unroll
                for (int r = 0; r < RPW; ++r) {
                    if (checked && j0 + j >= t.first + warp + 8 * r) continue;
                    const float2 w2 = make_float2(w[r], w[r]);
                    o[r][c][0] = fma_x2(w2, make_float2(x.x, x.y), o[r][c][0]);
                    o[r][c][1] = fma_x2(w2, make_float2(x.z, x.w), o[r][c][1]);
                }
            }
        };
        if (!busy) continue;
        if (!careful) {
#pragma unroll 4
            for (int j = 0; j < kKeys; ++j) values(j, false);
        } else {
#pragma unroll 1
            for (int j = 0; j < kKeys; ++j) values(j, true);
        }
    }
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        float sum = l[r];
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if (warp + 8 * r >= t.n_q) continue;
        const int64_t qh = (t.q0 + warp + 8 * r) * a.heads + h;
        const bool parts = a.n_split > 1;
        float* out = parts ? a.part_o + (qh * a.n_split + split) * VD : static_cast<float*>(a.out) + qh * VD;
        const float f = parts ? 1.f : 1.f / sum;
#pragma unroll
        for (int c = 0; c < kVec; ++c)
            store4(out + (c * 32 + lane) * 4, make_float4(o[r][c][0].x * f, o[r][c][0].y * f, o[r][c][1].x * f,
                                                          o[r][c][1].y * f));
        if (lane != 0) continue;
        if (parts) *reinterpret_cast<float2*>(a.part_ml + (qh * a.n_split + split) * 2) = make_float2(m[r], sum);
        else if (a.lse != nullptr) a.lse[qh] = expanded_lse(m[r], sum);
    }
}

// Tiles of 8 RPW queries, with fewer to a warp in one that has few: it still takes the
// tile's loads, but less arithmetic and shared memory (three prompts of 1, 129 and 257
// queries: 174 us instead of 217).
template <int RPW, int VD>
__global__ void __launch_bounds__(256, 2) expanded_simt(const ExpandedArgs a) {
    extern __shared__ __align__(16) float smem[];
    const int h = (int)(blockIdx.x % a.heads);
    const int split = (int)(blockIdx.x / a.heads % a.n_split);
    // a sequence's longest tiles first
    const int64_t slot = gridDim.x / a.heads / a.n_split - 1 - blockIdx.x / a.heads / a.n_split;
    pdl_wait();
    pdl_trigger();
    ExpandedTile t;
    if (expanded_tile(a.b, slot, split, a.n_split, 8 * RPW, kKeys, t)) {
        if (t.n_q <= 8) simt_tile<1, VD>(a, t, h, split, smem);
        else if (RPW > 2 && t.n_q <= 16) simt_tile<2, VD>(a, t, h, split, smem);
        else simt_tile<RPW, VD>(a, t, h, split, smem);
    }
    // a thread to a sequence, in as many CTAs as that takes
    if (blockIdx.x <= (uint32_t)a.b.n_seq / 256)
        expanded_check(a.b, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256, a.err, 60);
}

// One warp per (query, head): the splits' sums weighted by their maxima.  A CTA has eight queries of a
// slot's tile, so that queries of refused sequences, or of none, have no warp: no split was
// written for them.  The offsets are read before the wait for the splits, whose CTAs began behind
// theirs.
template <int VD>
__global__ void __launch_bounds__(256) expanded_merge(const ExpandedArgs a, const int bq) {
    const int64_t unit = blockIdx.x / (bq / 8);
    const int at = (int)(blockIdx.x % (bq / 8)) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    ExpandedTile t;
    const bool any = expanded_tile(a.b, unit / a.heads, 0, 1, bq, kKeys, t);
    pdl_wait();
    pdl_trigger();
    if (!any || at >= t.n_q) return;
    const int64_t qh = (t.q0 + at) * a.heads + unit % a.heads;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + qh * a.n_split;
    const float* po = a.part_o + qh * a.n_split * VD;
    float top = -INFINITY;
    for (int s = 0; s < a.n_split; ++s) top = fmaxf(top, ml[s].x);
    float4 o[VD / 128] = {};
    float l = 0.f;
    for (int s = 0; s < a.n_split; ++s) {
        const float2 x = ml[s];
        if (x.x == -INFINITY && x.y == 0.f) continue;    // a split without a key that the query sees
        const float w = x.x == -INFINITY ? x.y : exp2f(x.x - top);
        l += x.y * w;
#pragma unroll
        for (int c = 0; c < VD / 128; ++c) {
            const float4 y = load4(po + s * VD + (c * 32 + lane) * 4);
            o[c].x = fmaf(y.x, w, o[c].x); o[c].y = fmaf(y.y, w, o[c].y);
            o[c].z = fmaf(y.z, w, o[c].z); o[c].w = fmaf(y.w, w, o[c].w);
        }
    }
    const float inv = 1.f / l;
    float* out = static_cast<float*>(a.out) + qh * VD;
#pragma unroll
    for (int c = 0; c < VD / 128; ++c)
        store4(out + (c * 32 + lane) * 4, make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv));
    if (lane == 0 && a.lse != nullptr) a.lse[qh] = expanded_lse(top, l);
}

template <int RPW, int VD>
cudaError_t launch_tiles(const ExpandedArgs& a, cudaStream_t st) {
    auto kern = expanded_simt<RPW, VD>;
    const int bytes = simt_smem_floats(8 * RPW, a.nope + a.rope, VD) * 4;
    cudaError_t e = ensure_dyn_smem((const void*)kern, bytes);
    if (e != cudaSuccess) return e;
    const int64_t grid = expanded_slots(a.b.n_q, a.b.n_seq, 8 * RPW) * a.heads * a.n_split;
    return launch_pdl(kern, dim3((unsigned)grid), dim3(256), (size_t)bytes, st, a);
}

template <int VD>
cudaError_t launch_simt(const ExpandedArgs& a, int bq, cudaStream_t st) {
    cudaError_t e = bq == 16   ? launch_tiles<2, VD>(a, st)
                    : bq == 32 ? launch_tiles<4, VD>(a, st)
                               : launch_tiles<8, VD>(a, st);
    if (e != cudaSuccess || a.n_split == 1) return e;
    const int64_t grid = expanded_slots(a.b.n_q, a.b.n_seq, bq) * a.heads * (bq / 8);
    return launch_pdl(expanded_merge<VD>, dim3((unsigned)grid), dim3(256), 0, st, a, bq);
}

// Queries of a tile: 16 or 32 where no sequence has more, else 64 (two prompts of 1 and
// 20 tokens behind 100 and 0 rows: 13.3 us with 32, 19.9 with 64; eight of up to 32
// behind up to 1,000: 234 and 331).
int tile_queries(const BatchDev& b) { return b.max_q_len <= 16 ? 16 : b.max_q_len <= 32 ? 32 : kMaxTileQ; }

}  // namespace

// Splits of the key tiles: as many as end soonest, counting a wave of CTAs as
// its longest split and a split's partial sums as one more tile.
int32_t plan_expanded_splits(const Shape& sh, const BatchDev& b) {
    if (b.n_q < 1 || sh.dtype == DSA_BF16) return 1;
    const int64_t units = expanded_slots(b.n_q, b.n_seq, tile_queries(b)) * sh.heads;
    const int64_t wave = 2 * sm_count(), tiles = (b.max_kv_len + kKeys - 1) / kKeys;
    int32_t best = 1;
    int64_t least = INT64_MAX;
    for (int32_t s = 1; s <= kMaxSplit && s <= tiles && (s == 1 || units * s <= kSplitWaves * wave); ++s) {
        const int64_t cost = (units * s + wave - 1) / wave * ((tiles + s - 1) / s + (s > 1 ? 1 : 0));
        if (cost < least) { least = cost; best = s; }
    }
    return best;
}

// Room for every batch of no more queries, of sequences no longer: fewer queries
// may get more splits, but a tile's queries times its splits stay below the
// bound on a split call's CTAs.
size_t expanded_mla_scratch_bytes(const Shape& sh, const BatchDev& b) {
    if (sh.dtype == DSA_BF16 || b.max_kv_len <= kKeys) return 0;
    const int64_t most = kSplitWaves * 2 * sm_count() * kMaxTileQ / sh.heads;
    const int64_t all = (int64_t)b.n_q * kMaxSplit;
    return (size_t)(all < most ? all : most) * sh.heads * (256 + 2) * sizeof(float);
}

cudaError_t launch_expanded_mla(const Shape& sh, const BatchDev& b, int32_t nope, int32_t v_dim,
                                const void* q, const void* k_nope, const void* rows, const void* v,
                                void* out, float* lse, void* scratch, int32_t* err, cudaStream_t st) {
    if (b.n_q == 0) return cudaSuccess;
    ExpandedArgs a{};
    a.q = q; a.k_nope = k_nope; a.rows = rows; a.v = v; a.out = out; a.lse = lse;
    a.heads = sh.heads; a.nope = nope; a.rope = sh.rope; a.v_dim = v_dim; a.kv_lora = sh.kv_lora;
    a.width = sh.width(); a.scale = sh.scale; a.b = b; a.err = err;
    a.n_split = plan_expanded_splits(sh, b);
    a.part_o = static_cast<float*>(scratch);
    a.part_ml = a.part_o + (size_t)b.n_q * sh.heads * a.n_split * v_dim;
    if (sh.dtype == DSA_BF16) return launch_expanded_tc(a, st);
    const int bq = tile_queries(b);
    return v_dim == 256 ? launch_simt<256>(a, bq, st) : launch_simt<128>(a, bq, st);
}

}  // namespace dsa
