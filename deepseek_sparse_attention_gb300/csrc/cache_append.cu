// cache_append.cu -- new rows rounded into the paged 8-bit latent cache.
//
// For each page that a sequence's new rows fall in and each part of a row:
//     amax = the largest finite |x| of the new rows,
//     e    = the least integer with amax <= M 2^e (M = 448 for e4m3, 127 for
//            s8), kept within [-110, 119]; where the page holds earlier rows of
//            the sequence, at least the page's present exponent,
//     code = x / 2^e rounded to nearest even (to +-M beyond it),
// and where the exponent rose the earlier rows' codes are rounded again to it.
// Dividing by a power of two is exact, so each value is rounded once per
// exponent its page has had, and an e4m3 code that stays normal not at all
// when its page moves.
//
// One CTA per (sequence, page): no page is shared, so nothing is atomic.  The
// rows pass once: they stay in registers between the maximum and the rounding
// (the CTA is sized so that a page of up to 64 rows does; the rest of a larger
// one is read again), and are requested before the slots are read: a CTA's time
// is the latencies that it waits for in turn.  Bound by HBM for a prompt (2 or 4
// bytes read and one written per element; 183,000 float32 rows: 88 us = 0.79 of
// the measured bandwidth, 108 us with the slots first, 160 us in CTAs of 512
// threads whatever the page), by latency for a decode step (2.6 us for 64 rows).
#include "dsa_kernels.cuh"

namespace dsa {
namespace {

constexpr int kKeep = 9;               // vectors of 8 elements a thread keeps

struct Vec8 {
    float v[8];
};

template <typename T>
struct Raw;                            // 8 elements as loaded
template <>
struct Raw<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ Vec8 widen() const { return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
template <>
struct Raw<__nv_bfloat16> {
    uint4 w;
    __device__ void load(const __nv_bfloat16* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ Vec8 widen() const {
        Vec8 r;
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.v[2 * i] = __uint_as_float(u[i] << 16);
            r.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
        return r;
    }
};

template <int FMT>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
    if constexpr (FMT == DSA_CACHE_E4M3) {
        uint32_t r;                    // round to nearest even, +-448 beyond, NaN kept
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
        return r;
    } else {
        const float f[4] = {a, b, c, d};
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // fmaxf drops a NaN: handled here as 0
            const float x = f[i] == f[i] ? fminf(fmaxf(f[i], -127.f), 127.f) : 0.f;
            r |= ((uint32_t)__float2int_rn(x) & 0xffu) << (8 * i);
        }
        return r;
    }
}

// Least e with bits-as-float <= M 2^e, M = 1.75 * 2^8 (e4m3) or 1.984375 * 2^6
// (s8): the exponent of the value less that of M, one more when its mantissa
// exceeds M's.
template <int FMT>
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
    constexpr uint32_t mant = FMT == DSA_CACHE_E4M3 ? 0x600000u : 0x7e0000u;
    constexpr int shift = FMT == DSA_CACHE_E4M3 ? 8 : 6;
    const int e = (int)(bits >> 23) - 127 - shift + ((bits & 0x7fffffu) > mant ? 1 : 0);
    return min(max(e, kScaleExpMin), kScaleExpMax);
}

// grid: x = pages of one sequence's new rows, y = sequence.
template <typename T, int FMT, int W, int NT>
__global__ void __launch_bounds__(NT, 512 / NT)
cache_append_kernel(BatchDev b, PagesDev pg, const T* __restrict__ rows,
                    const int64_t* __restrict__ slots, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales, int32_t* err) {
    constexpr int kVecs = W / 8;                       // vectors of a row
    constexpr int kLatentVecs = kLatentCols / 8;
    constexpr int kParts = W > kLatentCols ? 2 : 1;
    __shared__ uint32_t s_max[2];
    __shared__ int s_bad;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int s = blockIdx.y;
    const int64_t q0 = b.q_off[s], q1 = b.q_off[s + 1];
    const int64_t kv = b.row_off[s + 1] - b.row_off[s], q_len = q1 - q0;
    if (q0 < 0 || q_len < 0 || q1 > b.n_q || q_len > kv || q_len > b.max_q_len ||
        kv > b.max_kv_len) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_error(err, kDevBadBatch, s, /*where=*/32);
        return;
    }
    const int64_t base = kv - q_len;                   // rows held before
    const int64_t c = (base >> pg.shift) + blockIdx.x; // the sequence's page
    const int64_t lo = max(base, c << pg.shift), hi = min(kv, (c + 1) << pg.shift);
    if (lo >= hi) return;
    const int n_new = (int)(hi - lo), off = (int)(lo & (pg.page_rows - 1));
    const int64_t tok = q0 + lo - base;
    const T* src = rows + tok * W;
    const int total = n_new * kVecs;
    Raw<T> keep[kKeep];
    const int64_t slot = slots[tok];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = threadIdx.x + k * NT;
        if (i < total) keep[k].load(src + (int64_t)i * 8);
    }
    if (threadIdx.x == 0) { s_max[0] = 0; s_max[1] = 0; s_bad = 0; }
    __syncthreads();
    if (slot == -1) return;                            // no page was planned for these rows
    // the page, and that its slots run on from the first one
    bool bad = slot < 0 || (slot >> pg.shift) >= pg.n_pages || (slot & (pg.page_rows - 1)) != off;
    for (int r = threadIdx.x; r < n_new; r += NT) bad |= slots[tok + r] != slot + r;

    // the largest finite magnitude of each part
    uint32_t mx[2] = {0, 0};
    bool odd = false;                                  // an infinity or a NaN
    auto fold = [&](int i, const Raw<T>& raw) {
        const Vec8 x = raw.widen();
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t a = __float_as_uint(x.v[k]) & 0x7fffffffu;
            const bool fin = a < 0x7f800000u;
            odd |= !fin;
            m = max(m, fin ? a : 0u);
        }
        if (kParts == 1 || i % kVecs < kLatentVecs) mx[0] = max(mx[0], m);
        else mx[1] = max(mx[1], m);
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = threadIdx.x + k * NT;
        if (i < total) fold(i, keep[k]);
    }
    for (int i = threadIdx.x + kKeep * NT; i < total; i += NT) {
        Raw<T> raw;
        raw.load(src + (int64_t)i * 8);
        fold(i, raw);
    }
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, mx[p]);
        if ((threadIdx.x & 31) == 0) atomicMax(&s_max[p], m);
    }
    if (bad) s_bad = 1;
    __syncthreads();
    if (s_bad) {
        if (threadIdx.x == 0) record_error(err, kDevBadIndex, s, /*where=*/32);
        return;
    }
    if (odd) record_error(err, kDevBadValue, s, /*where=*/32);
    uint8_t* page_scales = scales + (slot >> pg.shift) * kParts;
    int e_old[2] = {kScaleExpMin, kScaleExpMin}, e[2] = {0, 0};
    bool over = false;                                 // a scale the append never writes
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
        e[p] = scale_exponent<FMT>(s_max[p]);
        if (off > 0) {
            e_old[p] = (int)page_scales[p] - 127;
            over |= e_old[p] > kScaleExpMax;
            e[p] = max(e[p], e_old[p]);
        }
    }
    if (over) {
        if (threadIdx.x == 0) record_error(err, kDevBadValue, s, /*where=*/32);
        return;
    }
    __syncthreads();                                   // every thread has read the old scales
    if (threadIdx.x == 0) {
#pragma unroll
        for (int p = 0; p < kParts; ++p) page_scales[p] = (uint8_t)(e[p] + 127);
    }

    // the codes
    uint8_t* dst = codes + slot * W;
    auto put = [&](int i, const Raw<T>& raw) {
        const Vec8 x = raw.widen();
        const float f = exp2i(-(kParts == 1 || i % kVecs < kLatentVecs ? e[0] : e[1]));
        uint2 w;
        w.x = code4<FMT>(x.v[0] * f, x.v[1] * f, x.v[2] * f, x.v[3] * f);
        w.y = code4<FMT>(x.v[4] * f, x.v[5] * f, x.v[6] * f, x.v[7] * f);
        *reinterpret_cast<uint2*>(dst + (int64_t)i * 8) = w;
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = threadIdx.x + k * NT;
        if (i < total) put(i, keep[k]);
    }
    for (int i = threadIdx.x + kKeep * NT; i < total; i += NT) {
        Raw<T> raw;
        raw.load(src + (int64_t)i * 8);
        put(i, raw);
    }
    // earlier rows of the page whose exponent rose
    if (off > 0 && (e[0] > e_old[0] || (kParts == 2 && e[1] > e_old[1]))) {
        uint8_t* old = dst - (int64_t)off * W;
        for (int i = threadIdx.x; i < off * kVecs; i += NT) {
            const bool first = kParts == 1 || i % kVecs < kLatentVecs;
            const int d = first ? e_old[0] - e[0] : e_old[1] - e[1];
            if (d == 0) continue;
            const float f = exp2i(d);
            uint2 w = *reinterpret_cast<const uint2*>(old + (int64_t)i * 8);
            float x[4], y[4];
            widen_codes<FMT>(w.x, x);
            widen_codes<FMT>(w.y, y);
            w.x = code4<FMT>(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
            w.y = code4<FMT>(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
            *reinterpret_cast<uint2*>(old + (int64_t)i * 8) = w;
        }
    }
}

template <typename T, int FMT, int W>
cudaError_t launch_t(const BatchDev& b, const PagesDev& pg, const void* rows, const int64_t* slots,
                     uint8_t* codes, uint8_t* scales, int32_t* err, cudaStream_t st) {
    // pages a sequence's new rows can touch
    const int64_t gx = ((int64_t)b.max_q_len + pg.page_rows - 2) / pg.page_rows + 1;
    if (gx > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)gx, (unsigned)b.n_seq);
    // threads that keep all of a page's new rows in registers
    const int rows_max = b.max_q_len < pg.page_rows ? b.max_q_len : pg.page_rows;
    const int nt = (rows_max * (W / 8) + kKeep - 1) / kKeep;
    auto kern = nt <= 128   ? cache_append_kernel<T, FMT, W, 128>
                : nt <= 256 ? cache_append_kernel<T, FMT, W, 256>
                            : cache_append_kernel<T, FMT, W, 512>;
    const int threads = nt <= 128 ? 128 : nt <= 256 ? 256 : 512;
    return launch_pdl(kern, grid, dim3(threads), 0, st, b, pg, static_cast<const T*>(rows),
                      slots, codes, scales, err);
}

}  // namespace

cudaError_t launch_cache_append(const Shape& sh, const BatchDev& b, const PagesDev& pg,
                                const void* rows, const int64_t* slots, uint8_t* codes,
                                uint8_t* scales, int32_t* err, cudaStream_t st) {
    using bf16 = __nv_bfloat16;
    const bool f32 = sh.dtype == DSA_F32, wide = sh.width() == 576;
    auto f = pg.format == DSA_CACHE_E4M3
        ? (f32 ? (wide ? launch_t<float, DSA_CACHE_E4M3, 576> : launch_t<float, DSA_CACHE_E4M3, 512>)
               : (wide ? launch_t<bf16, DSA_CACHE_E4M3, 576> : launch_t<bf16, DSA_CACHE_E4M3, 512>))
        : (f32 ? (wide ? launch_t<float, DSA_CACHE_S8, 576> : launch_t<float, DSA_CACHE_S8, 512>)
               : (wide ? launch_t<bf16, DSA_CACHE_S8, 576> : launch_t<bf16, DSA_CACHE_S8, 512>));
    return f(b, pg, rows, slots, codes, scales, err, st);
}

}  // namespace dsa
