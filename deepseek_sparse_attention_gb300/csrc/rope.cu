// rope.cu -- rotary position embedding of part of each head, in place or from
// one tensor into another, in the adjacent-pair or the half layout.
//
//   angle = pos * rate_i,  (a, b) -> m (a cos - b sin, a sin + b cos)
//
// A pair is the columns (2i, 2i + 1) or (i, i + dims / 2).  The angle is formed
// in turns with integers, as for the indexer's rope: rate_i / 2 pi as a 64-bit
// binary fraction (made once, by dsa_rope_init) times the position, wrapping,
// which is exact modulo whole turns at any position.
//
// HBM-bound.  A thread has the same 16 bytes' worth of pairs (VEC) in several
// heads of one token, so that it makes each sine and cosine once for all of
// them; without the alignment for that it has one pair.
#include <math.h>

#include "dsa_kernels.cuh"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kThreads = 256;

struct RopeArgs {
    int64_t n_tok, x_tok, x_head, out_tok, out_head;
    const void* x;
    const int64_t* pos;
    void* out;
    int32_t heads, dims, inverse;
    float magnitude;
    int32_t units;         // threads along a head's pairs
    int32_t slots;         // threads along a token's heads
    int32_t tokens;        // tokens of a CTA
};
struct RopeTurns {
    unsigned long long r[DSA_ROPE_MAX_PAIRS];
};

__device__ __forceinline__ void round_to(float* d, float v) { *d = v; }
__device__ __forceinline__ void round_to(__nv_bfloat16* d, float v) { *d = __float2bfloat16_rn(v); }

// HPT heads of a token to a thread
template <typename T, bool HALVES, bool VEC, int HPT>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const RopeArgs a, const __grid_constant__ RopeTurns turns) {
    constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;     // elements of one move
    constexpr int kMoves = VEC && !HALVES ? 1 : 2;       // moves that hold a thread's pairs
    constexpr int kPairs = E * kMoves / 2;
    // into shared memory: lanes read different entries
    __shared__ unsigned long long turn[DSA_ROPE_MAX_PAIRS];
    const int half = a.dims / 2;
    for (int i = threadIdx.x; i < half; i += kThreads) turn[i] = turns.r[i];
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int per_token = a.units * a.slots;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    for (int w = threadIdx.x; w < a.tokens * per_token; w += kThreads) {
        const int64_t t = t0 + w / per_token;
        if (t >= a.n_tok) return;
        const int slot = w % per_token / a.units, u = w % a.units;
        // the thread's first column, and where its second move lies
        const int c0 = HALVES ? u * E : u * E * kMoves;
        const int step = HALVES ? half : 1;
        const T* x = static_cast<const T*>(a.x) + t * a.x_tok + c0;
        T* out = static_cast<T*>(a.out) + t * a.out_tok + c0;
        alignas(16) T v[HPT][kMoves][E];
#pragma unroll
        for (int k = 0; k < HPT; ++k) {
            const int h = slot + k * a.slots;
            if (h >= a.heads) break;
#pragma unroll
            for (int m = 0; m < kMoves; ++m) {
                if constexpr (VEC)
                    *reinterpret_cast<uint4*>(v[k][m]) =
                        *reinterpret_cast<const uint4*>(x + h * a.x_head + m * step);
                else
                    v[k][m][0] = x[h * a.x_head + m * step];
            }
        }
        const unsigned long long p = (unsigned long long)a.pos[t];
        float sn[kPairs], cs[kPairs];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int pair = HALVES ? c0 + i : c0 / 2 + i;
            // whole turns wrap away; the rest as a signed fraction of a half turn
            const int frac = (int)(unsigned int)((p * turn[pair]) >> 32);
            // bf16: the fast forms, within 2^-21.41 (sine) and 2^-21.19 (cosine) on [-pi, pi] of an
            // angle that three roundings leave within 5.7e-7: 1e-6 in all, far below bf16's
            // rounding (2^-8 of a value).  Float32: one rounding of the angle, 1.9e-7.
            if constexpr (sizeof(T) == 2)
                __sincosf((float)frac * 1.4629180792671596e-09f, &sn[i], &cs[i]);   // 2 pi / 2^32
            else
                sincospif((float)frac * 0x1p-31f, &sn[i], &cs[i]);
            if (a.inverse) sn[i] = -sn[i];
            sn[i] *= a.magnitude;
            cs[i] *= a.magnitude;
        }
#pragma unroll
        for (int k = 0; k < HPT; ++k) {
            const int h = slot + k * a.slots;
            if (h >= a.heads) break;
            alignas(16) T y[kMoves][E];
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                T *ya, *yb;
                float xa, xb;
                if constexpr (VEC && !HALVES) {
                    xa = to_float(v[k][0][2 * i]); xb = to_float(v[k][0][2 * i + 1]);
                    ya = &y[0][2 * i]; yb = &y[0][2 * i + 1];
                } else {
                    xa = to_float(v[k][0][i]); xb = to_float(v[k][kMoves - 1][i]);
                    ya = &y[0][i]; yb = &y[kMoves - 1][i];
                }
                round_to(ya, xa * cs[i] - xb * sn[i]);
                round_to(yb, xa * sn[i] + xb * cs[i]);
            }
#pragma unroll
            for (int m = 0; m < kMoves; ++m) {
                if constexpr (VEC)
                    *reinterpret_cast<uint4*>(out + h * a.out_head + m * step) =
                        *reinterpret_cast<const uint4*>(y[m]);
                else
                    out[h * a.out_head + m * step] = y[m][0];
            }
        }
    }
}

template <typename T, bool HALVES, bool VEC, int HPT>
cudaError_t launch(RopeArgs a, const RopeTurns& turns, cudaStream_t st) {
    a.slots = (a.heads + HPT - 1) / HPT;
    const int64_t per_token = (int64_t)a.units * a.slots;
    a.tokens = per_token >= kThreads ? 1 : (int32_t)(kThreads / per_token);
    const int64_t blocks = (a.n_tok + a.tokens - 1) / a.tokens;
    return launch_pdl(rope_kernel<T, HALVES, VEC, HPT>, dim3((unsigned)blocks), dim3(kThreads), 0, st,
                      a, turns);
}

template <typename T, bool HALVES>
cudaError_t launch(RopeArgs a, const RopeTurns& turns, cudaStream_t st) {
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t e = sizeof(T);
    auto fits = [&](const void* p, int64_t tok, int64_t head) {
        return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(tok * e) |
                 (a.heads > 1 ? (uintptr_t)(head * e) : 0)) & 15) == 0;
    };
    const int per = HALVES ? 2 * E : E;                  // columns of a thread's moves
    const bool vec = a.dims % per == 0 && fits(a.x, a.x_tok, a.x_head) && fits(a.out, a.out_tok, a.out_head);
    a.units = vec ? a.dims / per : a.dims / 2;
    // several heads to a thread, once that leaves every multiprocessor half full: two
    // heads 14.7 us for a 4,096-token chunk's queries, four 12.2, eight 12.4 (out of memory).
    // Several tokens of one head: 131,071 float32 tails 14.0 us with one, 14.5 with two.
    const bool many = a.n_tok * a.heads * a.units >= (int64_t)sm_count() * 2048 * 2;
    if (vec) return many && a.heads >= 4 ? launch<T, HALVES, true, 4>(a, turns, st)
                                         : launch<T, HALVES, true, 1>(a, turns, st);
    return many && a.heads >= 4 ? launch<T, HALVES, false, 4>(a, turns, st)
                                : launch<T, HALVES, false, 1>(a, turns, st);
}

}  // namespace

void init_rope_plan(int32_t dims, double base, double factor, double original_len, double beta_fast,
                    double beta_slow, uint64_t* turns) {
    const double two_pi = 6.283185307179586;
    // the pair that makes `n` turns over the trained context
    auto place = [&](double n) { return dims * log(original_len / (two_pi * n)) / (2.0 * log(base)); };
    double low = 0.0, high = -1.0;
    if (factor != 1.0 && beta_fast > 0.0) {
        low = floor(place(beta_fast));
        high = ceil(place(beta_slow));
        if (low < 0.0) low = 0.0;
        if (high > dims - 1.0) high = dims - 1.0;
    }
    for (int i = 0; i < dims / 2; ++i) {
        double rate = pow(base, -2.0 * i / (double)dims);
        if (factor != 1.0) {
            double g = 1.0;                              // how far the pair's rate is stretched
            if (beta_fast > 0.0) {
                const double span = high - low > 0.001 ? high - low : 0.001;
                g = (i - low) / span;
                g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            }
            rate *= (1.0 - g) + g / factor;
        }
        turns[i] = (uint64_t)nearbyint(ldexp(rate / two_pi, 64));
    }
}

cudaError_t launch_rope(const dsa_rope_plan& r, int32_t dtype, int64_t n_tok, int32_t heads,
                        const void* x, int64_t x_tok, int64_t x_head, const int64_t* pos, void* out,
                        int64_t out_tok, int64_t out_head, cudaStream_t st) {
    if (n_tok == 0 || heads == 0) return cudaSuccess;
    RopeTurns turns;
    for (int i = 0; i < DSA_ROPE_MAX_PAIRS; ++i) turns.r[i] = r.turns[i];
    RopeArgs a{};
    a.n_tok = n_tok; a.x_tok = x_tok; a.x_head = x_head; a.out_tok = out_tok; a.out_head = out_head;
    a.x = x; a.pos = pos; a.out = out;
    a.heads = heads; a.dims = r.dims; a.inverse = r.inverse; a.magnitude = r.magnitude;
    const bool halves = r.layout == DSA_ROPE_HALVES;
    if (dtype == DSA_BF16)
        return halves ? launch<__nv_bfloat16, true>(a, turns, st) : launch<__nv_bfloat16, false>(a, turns, st);
    return halves ? launch<float, true>(a, turns, st) : launch<float, false>(a, turns, st);
}

}  // namespace dsa
