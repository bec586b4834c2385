// rms_norm.cu -- root-mean-square norm of rows, with the residual's addition
// before it and an output in the rows' type or in 8 bits with scales.
//
//   h = x + add,   y = h / sqrt(mean(h^2) + eps) * weight
//   8 bits: scale_g = max(max_{j in g} |y_j| / 448, 2^-126), code_j = y_j / scale_g
//
// HBM-bound: a row is read once into registers, reduced and written.  It
// belongs to TPR threads; each of their warps takes chunks of 256 columns, a
// lane eight of them: neighbours, moved as 16 bytes, where pointers and strides
// allow it (VEC), else every 32nd, so that a warp's accesses of single elements
// are contiguous.  Either way the columns of a scale lie in one warp's chunk,
// and their maximum is a shuffle.  Where inputs alone are not aligned for it (rows an odd
// stride apart, say) and the output is codes, the aligned 16 bytes around each piece are
// read and shifted into place (SHIFT).
#include <cuda_fp8.h>

#include "dsa_kernels.cuh"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kPer = 8;                      // columns a lane has of a chunk
constexpr int kChunk = 32 * kPer;            // columns of a warp's chunk
constexpr float kTop = 448.f;                // the largest e4m3 value
constexpr float kLeast = 0x1p-126f;          // the least scale: its inverse is finite
constexpr float kMost = 3.402823466e38f;     // float32's largest value

// Eight elements as they are in memory: neighbours (VEC) or 32 apart.
template <typename T, bool VEC>
struct Raw;
template <bool VEC>
struct Raw<float, VEC> {
    float v[kPer];
    __device__ __forceinline__ float2 pair(int i) const { return make_float2(v[2 * i], v[2 * i + 1]); }
    __device__ __forceinline__ void set(int i, float2 x) { v[2 * i] = x.x; v[2 * i + 1] = x.y; }
};
template <>
struct Raw<__nv_bfloat16, true> {
    uint32_t v[kPer / 2];
    __device__ __forceinline__ float2 pair(int i) const {
        return make_float2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
    }
    __device__ __forceinline__ void set(int i, float2 x) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(x.x, x.y);
        v[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
};
template <>
struct Raw<__nv_bfloat16, false> {
    __nv_bfloat16 v[kPer];
    __device__ __forceinline__ float2 pair(int i) const {
        return make_float2(__bfloat162float(v[2 * i]), __bfloat162float(v[2 * i + 1]));
    }
    __device__ __forceinline__ void set(int i, float2 x) {
        v[2 * i] = __float2bfloat16_rn(x.x);
        v[2 * i + 1] = __float2bfloat16_rn(x.y);
    }
};

// ONCE: not kept in L1, where the weights shall stay.
template <bool ONCE, typename T, bool VEC>
__device__ __forceinline__ void load_chunk(Raw<T, VEC>& r, const T* p, int col, int width) {
    if constexpr (VEC) {
        if (col >= width) return;
        constexpr int n = sizeof(r) / 16;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint4* q = reinterpret_cast<const uint4*>(p + col) + i;
            uint4& x = reinterpret_cast<uint4*>(&r)[i];
            if constexpr (ONCE)
                asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                             : "l"(q)
                             : "memory");
            else
                x = *q;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (col + 32 * e < width) r.v[e] = p[col + 32 * e];
    }
}

// The aligned 16-byte words around a lane's eight columns of a row that begins anywhere;
// what they hold beside the row is not read.
template <typename T>
struct Around {
    static constexpr int kWords = kPer * sizeof(T) / 4 + 4;
    uint32_t w[kWords];
};
template <typename T>
__device__ __forceinline__ void load_around(Around<T>& r, const T* row, int col, int width) {
    const T* end = row + width;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15);
    const T* p = reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(row + col) - off);
#pragma unroll
    for (int g = 0; g < Around<T>::kWords / 4; ++g) {
        constexpr int n = 16 / sizeof(T);
        const T* q = p + g * n;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (col < width && (off != 0 || g + 1 < Around<T>::kWords / 4)) {
            if (q >= row && q + n <= end) {
                x = *reinterpret_cast<const uint4*>(q);
            } else {                                     // the row's first or last columns
                alignas(16) T e[n];
#pragma unroll
                for (int i = 0; i < n; ++i) e[i] = q + i >= row && q + i < end ? q[i] : T(0.f);
                x = *reinterpret_cast<const uint4*>(e);
            }
        }
        r.w[4 * g] = x.x; r.w[4 * g + 1] = x.y; r.w[4 * g + 2] = x.z; r.w[4 * g + 3] = x.w;
    }
}
template <typename T>
__device__ __forceinline__ void shift_in(Raw<T, true>& r, Around<T>& a, const T* row) {
    constexpr int n = kPer * sizeof(T) / 4;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15);
    if (off & 8)
#pragma unroll
        for (int i = 0; i < n + 2; ++i) a.w[i] = a.w[i + 2];
    if (off & 4)
#pragma unroll
        for (int i = 0; i < n + 1; ++i) a.w[i] = a.w[i + 1];
    uint32_t* out = reinterpret_cast<uint32_t*>(r.v);
#pragma unroll
    for (int i = 0; i < n; ++i) out[i] = sizeof(T) == 2 ? __funnelshift_r(a.w[i], a.w[i + 1], 8 * (off & 3)) : a.w[i];
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_chunk(T* p, const float2 (&h)[kPer / 2], int col, int width) {
    alignas(16) Raw<T, VEC> r;
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) r.set(i, h[i]);
    if constexpr (VEC) {
        if (col >= width) return;
        constexpr int n = sizeof(r) / 16;
#pragma unroll
        for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(p + col)[i] = reinterpret_cast<const uint4*>(&r)[i];
    } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (col + 32 * e < width) p[col + 32 * e] = r.v[e];
    }
}

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sum (or maximum) over the TPR threads of a row, the same in each of them.
// Rows of more than a warp have a CTA to themselves, so all its threads come here.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? max_nan(v, u) : v + u;
    }
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        v = buf[threadIdx.x % (TPR / 32)];               // the warps' values, several times over
#pragma unroll
        for (int o = TPR / 64; o > 0; o >>= 1) {
            const float u = __shfl_xor_sync(0xffffffffu, v, o);
            v = MAX ? max_nan(v, u) : v + u;
        }
    }
    return v;
}

// The steps from a product with an inverse to the quotient, below: q + (y - q s) / s, whose
// difference is exact ("Computation of elementary functions on the IBM RISC System/6000 processor",
// Markstein, 1990).  From amax / 448 it gives the rounded quotient for each of the 2^23 mantissas.
__device__ __forceinline__ float scale_of(float amax) {
    const float q = amax * (1.f / kTop);
    return max_nan(fmaf(fmaf(-fminf(q, kMost), kTop, amax), 1.f / kTop, q), kLeast);
}
// Two quotients y / s from r = 1 / s within a unit in the last place, rounded to float32 or, seldom, to
// its neighbour.  Their codes are those of the rounded quotients: over every mantissa of a scale and
// the nine y around each middle between two codes, a quotient is on its side of the middle, where
// the product alone is on another for 6.5%.  (Of a scale below 2^-92 the difference may lose bits; the
// quotient is then within 2^-22.  Keeping them by a power of two costs another product: 4,096 x
// 8,192 with residual 42.4 us, 41.4 so, 40.2 without the step.)
__device__ __forceinline__ float2 quotients(float2 y, float2 minus_s, float2 r) {
    const float2 q = mul_x2(y, r);
    return fma_x2(fma_x2(q, minus_s, y), r, q);
}
// The scale's part of them.  An infinite scale has finite quotients of zero.
__device__ __forceinline__ void divide_by(float s, float& minus_s, float& r) {
    minus_s = -fminf(s, kMost);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
}

// CTAs of a multiprocessor that the registers of a row and of the next one allow;
// 0: the next row is not asked for ahead, and rows have CTAs of their own.
template <typename T, bool VEC, int TPR, int C>
constexpr int kCtas = !VEC ? 0 : (C == 4 ? 512 : sizeof(T) == 2 ? 1024 : 768) / (TPR == 32 ? 256 : TPR);

// TPR threads to a row, each with up to C chunks' pieces; rows a stride apart, the
// next one's loads in flight while a row is reduced and written.
template <typename T, bool E4M3, bool VEC, bool SHIFT, int TPR, int C>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR,
                                  kCtas<T, VEC && !SHIFT, TPR, C> > 0 ? kCtas<T, VEC && !SHIFT, TPR, C> : 1)
rms_norm_kernel(const NormArgs a) {
    constexpr int kAhead = kCtas<T, VEC && !SHIFT, TPR, C>;
    constexpr int kRows = TPR == 32 ? 8 : 1;             // rows of a CTA
    constexpr int kWarps = TPR / 32;                     // warps of a row
    __shared__ float bufs[2][3][kWarps];
    const int lane = threadIdx.x & 31;
    const int warp = TPR == 32 ? 0 : threadIdx.x >> 5;
    const int64_t stride = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + (TPR == 32 ? threadIdx.x >> 5 : 0);
    if (row >= a.n_rows) return;
    pdl_wait();
    pdl_trigger();

    // this lane's first column of chunk c; its others follow (VEC) or are 32 apart
    auto col = [&](int c) { return (c * kWarps + warp) * kChunk + lane * (VEC ? kPer : 1); };
    alignas(16) Raw<T, VEC> rx[C], ra[C];
#pragma unroll
    for (int c = 0; c < C; ++c) rx[c] = ra[c] = Raw<T, VEC>{};
    auto fetch = [&](int64_t r) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_ld;
        if constexpr (SHIFT) {
            const T* add = a.add == nullptr ? nullptr : static_cast<const T*>(a.add) + r * a.add_ld;
            Around<T> wx[C], wa[C];
#pragma unroll
            for (int c = 0; c < C; ++c) load_around(wx[c], x, col(c), a.width);
            if (add != nullptr)
#pragma unroll
                for (int c = 0; c < C; ++c) load_around(wa[c], add, col(c), a.width);
#pragma unroll
            for (int c = 0; c < C; ++c) shift_in(rx[c], wx[c], x);
            if (add != nullptr)
#pragma unroll
                for (int c = 0; c < C; ++c) shift_in(ra[c], wa[c], add);
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) load_chunk<true>(rx[c], x, col(c), a.width);
            if (a.add == nullptr) return;
            const T* add = static_cast<const T*>(a.add) + r * a.add_ld;
#pragma unroll
            for (int c = 0; c < C; ++c) load_chunk<true>(ra[c], add, col(c), a.width);
        }
    };
    fetch(row);
    for (int turn = 0; row < a.n_rows; row += stride, turn ^= 1) {
        // other words than the row before: a warp may still read those
        float (&buf)[3][kWarps] = bufs[turn];
        float2 h[C][kPer / 2], sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) {
                h[c][i] = add_x2(rx[c].pair(i), ra[c].pair(i));   // zeros past the row
                sq = fma_x2(h[c][i], h[c][i], sq);
            }
        if (kAhead > 0 && row + stride < a.n_rows) {
            fetch(row + stride);
            // and the one after it into L2 (16-byte pieces, as the loads are)
            const int64_t later = row + 2 * stride;
            if (warp == 0 && lane == 0 && later < a.n_rows) {
                const uint32_t bytes = (uint32_t)a.width * sizeof(T);
                prefetch_l2_bytes(static_cast<const T*>(a.x) + later * a.x_ld, bytes);
                if (a.add != nullptr) prefetch_l2_bytes(static_cast<const T*>(a.add) + later * a.add_ld, bytes);
            }
        }
        float ss = row_reduce<TPR, false>(sq.x + sq.y, buf[0]);
        float rstd;
        // Squares, or their mean and eps, beyond float32, or so small that they lose bits which
        // eps does not cover: once more, of h times a power of two (all threads of the row).  High:
        // of 16,384 squares of up to 2^128 each, times 2^-160, the sum is below 2^111; a root above
        // 2^126 has a subnormal inverse, within 2^-22 of itself.
        const float square = fmaf(ss, a.mean, a.eps);
        const bool high = isinf(square);
        const bool low = ss < 0x1p-60f * (float)a.width && a.eps < 0x1p-60f;
        if (high || low) {
            const float f = high ? 0x1p-80f : 0x1p60f;
            ss = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i)
                    ss = fmaf(h[c][i].y * f, h[c][i].y * f, fmaf(h[c][i].x * f, h[c][i].x * f, ss));
            ss = row_reduce<TPR, false>(ss, buf[1]);
            rstd = f * rsqrtf(ss * a.mean + a.eps * f * f);
        } else {
            rstd = rsqrtf(square);
        }
        if (a.total != nullptr) {
            T* t = static_cast<T*>(a.total) + row * a.total_ld;
#pragma unroll
            for (int c = 0; c < C; ++c) store_chunk<T, VEC>(t, h[c], col(c), a.width);
        }
        float amax = 0.f;
        const float2 rstd2 = make_float2(rstd, rstd);
#pragma unroll
        for (int c = 0; c < C; ++c) {                    // y in the place of h
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) h[c][i] = mul_x2(h[c][i], rstd2);
            if (a.weight != nullptr) {
                alignas(16) Raw<float, VEC> w;
#pragma unroll
                for (int e = 0; e < kPer; ++e) w.v[e] = 0.f;
                load_chunk<false>(w, a.weight, col(c), a.width);
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) h[c][i] = mul_x2(h[c][i], w.pair(i));
            }
            if (E4M3 && a.group == 0)
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) amax = max_nan(max_nan(amax, fabsf(h[c][i].x)), fabsf(h[c][i].y));
        }
        if constexpr (!E4M3) {
            T* y = static_cast<T*>(a.out) + row * a.out_ld;
#pragma unroll
            for (int c = 0; c < C; ++c) store_chunk<T, VEC>(y, h[c], col(c), a.width);
        } else {
            const int shift = a.group == 0 ? 30 : 31 - __clz(a.group);   // a column's scale: its number >> shift
            float* scales = a.scales + row * (((a.width - 1) >> shift) + 1);
            uint8_t* codes = static_cast<uint8_t*>(a.out) + row * a.out_ld;
            float s = 0.f;
            if (a.group == 0) {
                s = scale_of(row_reduce<TPR, true>(amax, buf[2]));
                if (warp == 0 && lane == 0) scales[0] = s;
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int at = (c * kWarps + warp) * kChunk;
                if (at >= a.width) break;                // the whole warp
                float2 minus_s[VEC ? 1 : kPer / 2], inv[VEC ? 1 : kPer / 2];
                if (VEC || a.group == 0) {
                    if (a.group != 0) {                  // 4, 8 or 16 lanes
                        float m = 0.f;
#pragma unroll
                        for (int i = 0; i < kPer / 2; ++i) m = max_nan(max_nan(m, fabsf(h[c][i].x)), fabsf(h[c][i].y));
                        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
                        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
                        if (shift > 5) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        if (shift > 6) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        s = scale_of(m);
                        if ((col(c) & (a.group - 1)) == 0 && col(c) < a.width) scales[col(c) >> shift] = s;
                    }
                    float ms, r;
                    divide_by(s, ms, r);
#pragma unroll
                    for (int i = 0; i < (VEC ? 1 : kPer / 2); ++i) {
                        minus_s[i] = make_float2(ms, ms);
                        inv[i] = make_float2(r, r);
                    }
                } else {                                 // 1, 2 or 4 neighbouring elements of all lanes
                    const int n = a.group / 32;
                    float m[kPer];
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        // as integers, which order as the numbers do, NaN above them
                        m[e] = __uint_as_float(__reduce_max_sync(
                            0xffffffffu, __float_as_uint(fabsf(e & 1 ? h[c][e / 2].y : h[c][e / 2].x))));
                    }
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        const float m2 = max_nan(m[e & ~1], m[e | 1]);
                        const float m4 = max_nan(max_nan(m[e & ~3], m[(e & ~3) + 1]),
                                                 max_nan(m[(e & ~3) + 2], m[e | 3]));
                        s = scale_of(n == 1 ? m[e] : n == 2 ? m2 : m4);
                        if (lane == 0 && e % n == 0 && at + 32 * e < a.width) scales[(at + 32 * e) >> shift] = s;
                        float2 &ms = minus_s[VEC ? 0 : e / 2], &r = inv[VEC ? 0 : e / 2];
                        divide_by(s, e & 1 ? ms.y : ms.x, e & 1 ? r.y : r.x);
                    }
                }
                // to nearest even; a NaN stays one
                alignas(8) uint8_t q[kPer];
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) {
                    const __nv_fp8x2_storage_t two = __nv_cvt_float2_to_fp8x2(
                        quotients(h[c][i], minus_s[VEC ? 0 : i], inv[VEC ? 0 : i]), __NV_SATFINITE, __NV_E4M3);
                    q[2 * i] = (uint8_t)(two & 0xff);
                    q[2 * i + 1] = (uint8_t)(two >> 8);
                }
                if (VEC) {
                    if (col(c) < a.width)
                        *reinterpret_cast<uint2*>(codes + col(c)) = *reinterpret_cast<const uint2*>(q);
                } else {
#pragma unroll
                    for (int e = 0; e < kPer; ++e)
                        if (col(c) + 32 * e < a.width) codes[col(c) + 32 * e] = q[e];
                }
            }
        }
    }
}

template <typename T, bool E4M3, bool VEC, bool SHIFT, int TPR, int C>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
    constexpr int kRows = TPR == 32 ? 8 : 1;
    int64_t blocks = (a.n_rows + kRows - 1) / kRows;
    const int64_t wave = (int64_t)sm_count() * kCtas<T, VEC && !SHIFT, TPR, C>;
    if (wave > 0 && blocks > wave) blocks = wave;
    return launch_pdl(rms_norm_kernel<T, E4M3, VEC, SHIFT, TPR, C>, dim3((unsigned)blocks),
                      dim3(TPR == 32 ? 256 : TPR), 0, st, a);
}

template <typename T, bool E4M3, bool VEC, bool SHIFT>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
    // a warp to a row of up to 1,024 columns; beyond, as many threads as leave each
    // two pieces of eight columns: its registers then let 1,500 threads or more of a
    // multiprocessor have loads in flight
    if (a.width <= 512) return launch<T, E4M3, VEC, SHIFT, 32, 2>(a, st);
    if (a.width <= 1024) return launch<T, E4M3, VEC, SHIFT, 32, 4>(a, st);
    if (a.width <= 2048) return launch<T, E4M3, VEC, SHIFT, 128, 2>(a, st);
    if (a.width <= 4096) return launch<T, E4M3, VEC, SHIFT, 256, 2>(a, st);
    if (a.width <= 8192) return launch<T, E4M3, VEC, SHIFT, 512, 2>(a, st);
    return launch<T, E4M3, VEC, SHIFT, 512, 4>(a, st);
}

enum class Access { kVec, kShift, kSingle };

template <typename T>
cudaError_t launch(const NormArgs& a, bool e4m3, Access how, cudaStream_t st) {
    if (how == Access::kShift) return launch<T, true, true, true>(a, st);
    if (e4m3) return how == Access::kVec ? launch<T, true, true, false>(a, st) : launch<T, true, false, false>(a, st);
    return how == Access::kVec ? launch<T, false, true, false>(a, st) : launch<T, false, false, false>(a, st);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int32_t dtype, bool e4m3, cudaStream_t st) {
    if (a.n_rows == 0) return cudaSuccess;
    // 16-byte moves (8 for codes) where every pointer, stride and the width allow them
    const int64_t e = dtype == DSA_BF16 ? 2 : 4;
    auto fits = [](const void* p, int64_t ld, int64_t size, int64_t unit) {
        return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * size)) & (unit - 1)) == 0;
    };
    const bool out = a.width % kPer == 0 && fits(a.total, a.total_ld, e, 16) && fits(a.weight, 0, 4, 16) &&
                     (e4m3 ? fits(a.out, a.out_ld, 1, 8) : fits(a.out, a.out_ld, e, 16));
    const bool in = fits(a.x, a.x_ld, e, 16) && fits(a.add, a.add_ld, e, 16);
    // shifted for codes alone, whose scales want neighbours in a lane: 3,400 bf16 rows of 8,192
    // columns, 8,195 apart, 49 us and one by one 92 (with a residual 121 and 122); to bf16 rows
    // 52 and 48
    const Access how = out && in ? Access::kVec : out && e4m3 ? Access::kShift : Access::kSingle;
    return dtype == DSA_BF16 ? launch<__nv_bfloat16>(a, e4m3, how, st) : launch<float>(a, e4m3, how, st);
}

}  // namespace dsa
