// expand_kv.cu -- the latent rows expanded into every head's keys and values.
//
//   k_nope[r, h, d] = sum_{i < kv_lora} w_uk[h, d, i] * latent[r, i]
//   v[r, h, e]      = sum_{i < kv_lora} w_uv[h, e, i] * latent[r, i]
//
// "GLM 5.2 in one C file", "Attention: Multi head Latent Attention With a Tiny
// KV Cache": the explicit form of what absorption folds into the query and the
// output.  Two matrix products of the rows [n_rows, kv_lora] with the weights
// [heads * d, kv_lora], both with the sum along contiguous memory, in one launch.
//
// bf16 runs on the tensor cores (expand_kv_tc.cu).  Float32, on CUDA cores: tiles of 64 rows
// by 128 outputs, 8 x 8 of them to a thread, 16 terms of the sum at a time through
// two buffers of shared memory, the next in flight in registers.  Bound by float32
// arithmetic: 300 rows to 64 heads' 192 + 256 columns take 176 us, 0.66 of that rate, of which
// a twelfth is the last tiles' idle multiprocessors.  Four CTAs of 128 threads to a
// multiprocessor (two of 256, tiles of 64 x 256: 180 us; three, which spares a spill of
// ten words: 189), 8 terms at a time 205, 8 x 16 to a thread 194.
#include "dsa_kernels.cuh"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kRows = 64, kCols = 128, kDepth = 16;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__global__ void __launch_bounds__(128, 4)
expand_simt(const float* __restrict__ rows, const float* __restrict__ w_uk, const float* __restrict__ w_uv,
            float* __restrict__ k_nope, float* __restrict__ v, int64_t n_rows, int32_t width, int32_t kv_lora,
            int32_t n_k, int32_t n_v) {
    // by term; a term's column is xored with 8 (term / 4), so that the lanes that hold four
    // terms each of the same row write to different banks (tiles of 64 x 256: 180 us, 196 without)
    __shared__ float As[2][kDepth][kRows], Bs[2][kDepth][kCols];
    const int tiles = (n_k + n_v) / kCols;
    const int64_t r0 = (int64_t)(blockIdx.x / tiles) * kRows;
    int n0 = (int)(blockIdx.x % tiles) * kCols;
    const bool is_v = n0 >= n_k;                         // both widths are multiples of a tile's
    if (is_v) n0 -= n_k;
    const float* w = is_v ? w_uv : w_uk;
    float* out = is_v ? v : k_nope;
    const int ld = is_v ? n_v : n_k;
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    // this thread's pieces of four terms: two of the rows, four of the weights, 32 lines apart
    const int line = t >> 2, k4 = (t & 3) * 4;
    const float* pa[2];
    bool has[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r = r0 + line + i * 32;
        has[i] = r < n_rows;
        pa[i] = rows + (has[i] ? r : 0) * width + k4;
    }
    const float* pb = w + (int64_t)(n0 + line) * kv_lora + k4;
    float4 a[2], b[4];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = has[i] ? load4(pa[i] + k0) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = load4(pb + (int64_t)i * 32 * kv_lora + k0);
    };
    auto put = [&](int buf) {
        const int sw = k4 * 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = (line + i * 32) ^ sw;
            As[buf][k4][n] = a[i].x; As[buf][k4 + 1][n] = a[i].y; As[buf][k4 + 2][n] = a[i].z; As[buf][k4 + 3][n] = a[i].w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = (line + i * 32) ^ sw;
            Bs[buf][k4][n] = b[i].x; Bs[buf][k4 + 1][n] = b[i].y; Bs[buf][k4 + 2][n] = b[i].z; Bs[buf][k4 + 3][n] = b[i].w;
        }
    };
    float acc[8][8] = {};
    load(0);
    put(0);
    __syncthreads();
    for (int k0 = 0, buf = 0; k0 < kv_lora; k0 += kDepth, buf ^= 1) {
        const bool more = k0 + kDepth < kv_lora;
        if (more) load(k0 + kDepth);
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            const int ra = (ty * 8) ^ (k / 4 * 8), cb = (tx * 4) ^ (k / 4 * 8);
            const float4 a0 = load4(&As[buf][k][ra]), a1 = load4(&As[buf][k][ra + 4]);
            const float4 b0 = load4(&Bs[buf][k][cb]), b1 = load4(&Bs[buf][k][64 + cb]);
            const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            const float bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 8; j += 2) fma2(acc[i][j], acc[i][j + 1], av[i], av[i], bv[j], bv[j + 1]);
        }
        if (more) put(buf ^ 1);                          // read by all before the last barrier
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + ty * 8 + i;
        if (r >= n_rows) continue;
        float* o = out + r * ld + n0 + tx * 4;
        store4(o, acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        store4(o + 64, acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
}

cudaError_t launch_simt(const Shape& sh, int64_t n_rows, int32_t nope, int32_t v_dim, const void* rows,
                        const void* w_uk, const void* w_uv, void* k_nope, void* v, cudaStream_t st) {
    const int32_t n_k = sh.heads * nope, n_v = sh.heads * v_dim;
    const int64_t grid = (n_rows + kRows - 1) / kRows * ((n_k + n_v) / kCols);
    return launch_plain(expand_simt, dim3((unsigned)grid), dim3(128), 0, st, static_cast<const float*>(rows),
                        static_cast<const float*>(w_uk), static_cast<const float*>(w_uv),
                        static_cast<float*>(k_nope), static_cast<float*>(v), n_rows, sh.width(), sh.kv_lora, n_k, n_v);
}

}  // namespace

cudaError_t launch_expand_kv(const Shape& sh, int64_t n_rows, int32_t nope, int32_t v_dim,
                             const void* rows, const void* w_uk, const void* w_uv, void* k_nope,
                             void* v, int32_t* err, cudaStream_t st) {
    if (n_rows == 0) return cudaSuccess;
    return sh.dtype == DSA_BF16
               ? launch_expand_tc(sh, n_rows, nope, v_dim, rows, w_uk, w_uv, k_nope, v, err, st)
               : launch_simt(sh, n_rows, nope, v_dim, rows, w_uk, w_uv, k_nope, v, st);
}

}  // namespace dsa
