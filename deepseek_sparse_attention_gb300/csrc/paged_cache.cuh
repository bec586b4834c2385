// paged_cache.cuh -- the paged 8-bit latent cache as the kernels see it.
//
// A pool of n_pages pages of page_rows rows each; a row is W = kv_lora + rope
// 8-bit codes.  Every page keeps one scale per part of a row (the latent, and
// the rope tail where there is one), an E8M0 byte b standing for 2^(b - 127):
// a code c stands for c * 2^(b - 127).  Scales are powers of two so that
// applying one, and moving a row to a larger one, rounds nothing but the code
// itself.  Row r of sequence s is row r % page_rows of page
// block_table[s][r / page_rows].
#pragma once

#include <cuda_fp16.h>

#include "dsa_common.cuh"

namespace dsa {

constexpr int kLatentCols = 512;       // columns of the first part of a row

// Exponents the append gives a page's scale: a code times it stays a normal
// float32 and bfloat16.
constexpr int kScaleExpMin = -110, kScaleExpMax = 119;

struct PagesDev {
    int32_t page_rows;
    int32_t shift;                     // log2(page_rows)
    int32_t format;                    // a dsa_cache_format
    int64_t n_pages;
    int64_t table_ld;
};

// Page of row r >= 0 of sequence s, or -1 when the table has no page there.
__device__ __forceinline__ int32_t page_of(const PagesDev& pg, const int32_t* block_table,
                                           int32_t s, int64_t r) {
    const int64_t c = r >> pg.shift;
    if (c >= pg.table_ld) return -1;
    const int32_t p = block_table[(int64_t)s * pg.table_ld + c];
    return p >= 0 && p < pg.n_pages ? p : -1;
}

// The power of two an E8M0 byte stands for (255: NaN).
__device__ __forceinline__ float e8m0(uint32_t b) {
    const uint32_t bits = b == 0u ? 0x00400000u : (b == 255u ? 0x7fffffffu : b << 23);
    return __uint_as_float(bits);
}

// 2^e for -126 <= e <= 127, exactly; 0 below.
__device__ __forceinline__ float exp2i(int e) {
    return e < -126 ? 0.f : __uint_as_float((uint32_t)(e + 127) << 23);
}

// The four codes of a word widened to float (exact in both formats).
template <int FMT>
__device__ __forceinline__ void widen_codes(uint32_t w, float (&f)[4]) {
    if constexpr (FMT == DSA_CACHE_E4M3) {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
    } else {
        // a byte b under the exponent of 2^23 reads 2^23 + b; with the sign bit
        // flipped b = code + 128, so subtracting 2^23 + 128 leaves the code
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440u + i)) - 8388736.f;
    }
}

// The four codes of a word as f16 (exact in both formats), two per word.
template <int FMT>
__device__ __forceinline__ uint2 codes_f16(uint32_t w) {
    uint2 r;
    if constexpr (FMT == DSA_CACHE_E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(r.x), "=r"(r.y) : "r"(w));
    } else {
        // a byte b under the exponent of 2^10 reads 1024 + b, b = code + 128
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));      // 1152
        const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), off);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
        r.x = *reinterpret_cast<const uint32_t*>(&a);
        r.y = *reinterpret_cast<const uint32_t*>(&b);
    }
    return r;
}

}  // namespace dsa
