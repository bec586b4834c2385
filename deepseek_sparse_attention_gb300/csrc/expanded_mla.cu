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
// One CTA per (tile of 16 RPT queries, head, split of the key tiles): one pass over
// tiles of 32 keys with a running maximum and sum.  16 lanes share a thread's
// RPT query rows: of the logits a thread has those rows and two keys, of the
// output the rows and every 16th group of four columns.  Bound by shared-memory
// reads (a logit's operands are used RPT and twice) and float32 arithmetic.
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

template <int RPT, int VD>
__global__ void __launch_bounds__(256, 2) expanded_simt(const ExpandedArgs a) {
    constexpr int BQ = 16 * RPT;
    constexpr int kVec = VD / 64;                        // groups of four output columns of a thread
    extern __shared__ __align__(16) float smem[];
    const int d = a.nope + a.rope, ld = d + 4;
    float* Qs = smem;
    float* Ks = Qs + BQ * ld;
    float* Vs = Ks;
    float* Ps = Ks + kKeys * (ld > VD ? ld : VD);        // [key][query], rows of BQ + 4

    const int h = (int)(blockIdx.x % a.heads);
    const int split = (int)(blockIdx.x / a.heads % a.n_split);
    const int64_t slot = blockIdx.x / a.heads / a.n_split;
    pdl_wait();
    pdl_trigger();
    ExpandedTile t;
    if (!expanded_tile(a.b, slot, split, a.n_split, BQ, kKeys, a.err, 60, t)) return;

    const float* q = static_cast<const float*>(a.q);
    const float* kn = static_cast<const float*>(a.k_nope);
    const float* rows = static_cast<const float*>(a.rows);
    const float* v = static_cast<const float*>(a.v);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = tid; i < BQ * d / 4; i += 256) {
        const int r = i / (d / 4), c = i % (d / 4) * 4;
        store4(Qs + r * ld + c, r < t.n_q ? load4(q + ((t.q0 + r) * a.heads + h) * d + c) : zero);
    }
    float o[RPT][kVec][4] = {};
    float m[RPT], l[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) { m[r] = -INFINITY; l[r] = 0.f; }
    const float scale = a.scale * kLog2e;
    const int64_t last = t.first + t.n_q - 1;            // rows that the tile's last query sees

    for (int kt = t.kt0; kt < t.kt1; ++kt) {
        const int64_t j0 = (int64_t)kt * kKeys;
        __syncthreads();
        for (int i = tid; i < kKeys * d / 4; i += 256) {
            const int j = i / (d / 4), c = i % (d / 4) * 4;
            const int64_t row = t.row0 + j0 + j;
            float4 x = zero;
            if (j0 + j < last)
                x = c < a.nope ? load4(kn + (row * a.heads + h) * a.nope + c)
                               : load4(rows + row * a.width + a.kv_lora + c - a.nope);
            store4(Ks + j * ld + c, x);
        }
        __syncthreads();
        float s[RPT][2] = {};
#pragma unroll 4
        for (int c = 0; c < d; c += 4) {
            const float4 k0 = load4(Ks + tx * ld + c), k1 = load4(Ks + (tx + 16) * ld + c);
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const float4 x = load4(Qs + (ty * RPT + r) * ld + c);
                s[r][0] = fmaf(x.x, k0.x, fmaf(x.y, k0.y, fmaf(x.z, k0.z, fmaf(x.w, k0.w, s[r][0]))));
                s[r][1] = fmaf(x.x, k1.x, fmaf(x.y, k1.y, fmaf(x.z, k1.z, fmaf(x.w, k1.w, s[r][1]))));
            }
        }
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            const int64_t sees = t.first + ty * RPT + r;
            const float s0 = j0 + tx < sees ? s[r][0] * scale : -INFINITY;
            const float s1 = j0 + tx + 16 < sees ? s[r][1] * scale : -INFINITY;
            float top = fmaxf(s0, s1);
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float mn = fmaxf(m[r], top);
            const float base = mn == -INFINITY ? 0.f : mn;   // nothing to see so far
            const float f = exp2f(m[r] - base);
            const float p0 = exp2f(s0 - base), p1 = exp2f(s1 - base);
            float sum = p0 + p1;
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            l[r] = l[r] * f + sum;
            m[r] = mn;
#pragma unroll
            for (int c = 0; c < kVec; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[r][c][e] *= f;
            Ps[tx * (BQ + 4) + ty * RPT + r] = p0;
            Ps[(tx + 16) * (BQ + 4) + ty * RPT + r] = p1;
        }
        __syncthreads();                                 // the keys are read
        for (int i = tid; i < kKeys * VD / 4; i += 256) {
            const int j = i / (VD / 4), c = i % (VD / 4) * 4;
            store4(Vs + j * VD + c, j0 + j < last ? load4(v + ((t.row0 + j0 + j) * a.heads + h) * VD + c) : zero);
        }
        __syncthreads();
        const bool all = j0 + kKeys <= t.first;          // every query sees every key of the tile
        auto values = [&](int j, bool checked) {
            float p[RPT];
            if constexpr (RPT == 4) {
                const float4 x = load4(Ps + j * (BQ + 4) + ty * 4);
                p[0] = x.x; p[1] = x.y; p[2] = x.z; p[3] = x.w;
            } else {
#pragma unroll
                for (int r = 0; r < RPT; ++r) p[r] = Ps[j * (BQ + 4) + ty * RPT + r];
            }
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                const float4 x = load4(Vs + j * VD + (c * 16 + tx) * 4);
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    // a hidden value may be anything: 0 times infinity is NaN
                    if (checked && j0 + j >= t.first + ty * RPT + r) continue;
                    fma2(o[r][c][0], o[r][c][1], p[r], p[r], x.x, x.y);
                    fma2(o[r][c][2], o[r][c][3], p[r], p[r], x.z, x.w);
                }
            }
        };
        if (all) {
#pragma unroll 4
            for (int j = 0; j < kKeys; ++j) values(j, false);
        } else {
            for (int j = 0; j < kKeys; ++j) values(j, true);
        }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int i = ty * RPT + r;
        if (i >= t.n_q) continue;
        const int64_t qh = (t.q0 + i) * a.heads + h;
        if (a.n_split > 1) {
            float* po = a.part_o + (qh * a.n_split + split) * VD;
#pragma unroll
            for (int c = 0; c < kVec; ++c)
                store4(po + (c * 16 + tx) * 4, make_float4(o[r][c][0], o[r][c][1], o[r][c][2], o[r][c][3]));
            if (tx == 0)
                *reinterpret_cast<float2*>(a.part_ml + (qh * a.n_split + split) * 2) = make_float2(m[r], l[r]);
        } else {
            float* out = static_cast<float*>(a.out) + qh * VD;
            const float inv = 1.f / l[r];
#pragma unroll
            for (int c = 0; c < kVec; ++c)
                store4(out + (c * 16 + tx) * 4, make_float4(o[r][c][0] * inv, o[r][c][1] * inv,
                                                            o[r][c][2] * inv, o[r][c][3] * inv));
            if (tx == 0 && a.lse != nullptr) a.lse[qh] = expanded_lse(m[r], l[r]);
        }
    }
}

// One warp per (query, head): the splits' sums weighted by their maxima.
template <int VD>
__global__ void __launch_bounds__(256) expanded_merge(const ExpandedArgs a, int64_t n) {
    const int64_t qh = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (qh >= n) return;
    pdl_wait();
    pdl_trigger();
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

template <int RPT, int VD>
cudaError_t launch_tiles(const ExpandedArgs& a, cudaStream_t st) {
    auto kern = expanded_simt<RPT, VD>;
    const int bytes = simt_smem_floats(16 * RPT, a.nope + a.rope, VD) * 4;
    cudaError_t e = ensure_dyn_smem((const void*)kern, bytes);
    if (e != cudaSuccess) return e;
    const int64_t grid = expanded_slots(a.b.n_q, a.b.n_seq, 16 * RPT) * a.heads * a.n_split;
    return launch_pdl(kern, dim3((unsigned)grid), dim3(256), (size_t)bytes, st, a);
}

template <int VD>
cudaError_t launch_simt(const ExpandedArgs& a, bool few, cudaStream_t st) {
    cudaError_t e = few ? launch_tiles<1, VD>(a, st) : launch_tiles<4, VD>(a, st);
    if (e != cudaSuccess || a.n_split == 1) return e;
    const int64_t n = (int64_t)a.b.n_q * a.heads;
    return launch_pdl(expanded_merge<VD>, dim3((unsigned)((n + 7) / 8)), dim3(256), 0, st, a, n);
}

// Queries of a tile: 16 where no sequence has more, else 64.
bool few_queries(const BatchDev& b) { return b.max_q_len <= 16; }

}  // namespace

// Splits of the key tiles: as many as end soonest, counting a wave of CTAs as
// its longest split and a split's partial sums as one more tile.
int32_t plan_expanded_splits(const Shape& sh, const BatchDev& b) {
    if (b.n_q < 1 || sh.dtype == DSA_BF16) return 1;
    const int64_t units = expanded_slots(b.n_q, b.n_seq, few_queries(b) ? 16 : 64) * sh.heads;
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
    const bool few = few_queries(b);
    return v_dim == 256 ? launch_simt<256>(a, few, st) : launch_simt<128>(a, few, st);
}

}  // namespace dsa
