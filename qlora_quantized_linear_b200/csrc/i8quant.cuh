// i8quant.cuh -- symmetric 8-bit quantization of matrix rows: one scale per
// row (per token of an activation, per output channel of a weight).
//
//   amax = max_j |v_j|,  scale = fp32(amax / 127),
//   code_j = 127 v_j / amax rounded to the nearest integer, ties to even.
//
// The codes are those of the exact quotient, so they do not depend on how a
// reciprocal rounds; bf16 data meets exact ties often (v = amax / 2 is 63.5).
// The fast path multiplies by fp32(127 / amax): its relative error is below
// 2^-22, so for |r| <= 127 the absolute error is below 2^-15 and the rounded
// value is right unless r lies within 2^-12 of a half-integer.  Those elements
// (one in about 2^11, and the ties) compare 127 v with the half-integer times
// amax in fp64, where both products are exact (24 + 8 bits).
//
// HBM-bound: a row is read once and stays in registers between its maximum and
// its codes.
// A zero row has scale 0 and codes 0.  A row that holds an infinity or a NaN
// has scale NaN and codes 0, so every product of the row is NaN.
#pragma once

#include "common.cuh"

namespace lbq {

enum I8Src : int { kSrcF32 = LBQ_F32, kSrcBf16 = LBQ_BF16, kSrcF16 = LBQ_F16 };

struct I8RowScale {
    float f;      // power of two applied to the values first (amax of a row of tiny values)
    float inv;    // fp32(127 / (amax f)); 0 for a row without codes
    float a;      // amax f
    float scale;  // the stored scale
};

__device__ __forceinline__ I8RowScale i8_row_scale(uint32_t amax_bits) {
    I8RowScale r;
    const float a = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7F800000u) {
        r = I8RowScale{0.0f, 0.0f, 1.0f, __uint_as_float(0x7FC00000u)};
    } else if (amax_bits == 0u) {
        r = I8RowScale{1.0f, 0.0f, 1.0f, 0.0f};
    } else {
        // 127 / amax overflows below 2^-121: such rows are brought up by 2^100 (exact)
        r.f = a < 8.6736174e-19f /* 2^-60 */ ? 1.2676506e30f /* 2^100 */ : 1.0f;
        r.a = a * r.f;
        r.inv = __fdiv_rn(127.0f, r.a);
        r.scale = __fdiv_rn(a, 127.0f);
    }
    return r;
}

// The code of one value (already multiplied by r.f) by the exact comparison.
__device__ __noinline__ int i8_code_exact(float v, float inv, float a) {
    const float x = v * inv;
    int c = __float2int_rn(x);
    if (fabsf(x - static_cast<float>(c)) > 0.5f - 0x1p-12f) {
        const float h = floorf(fabsf(x) + 0x1p-11f - 0.5f) + 0.5f;          // the half-integer next to |x|
        const double p = 127.0 * static_cast<double>(fabsf(v));
        const double t = static_cast<double>(h) * static_cast<double>(a);
        const int lo = static_cast<int>(h - 0.5f);
        const int m = p > t ? lo + 1 : p < t ? lo : lo + (lo & 1);
        c = v < 0.0f ? -m : m;
    }
    return c;
}

// The codes of eight values, first in the low byte.  v inv + 1.5 * 2^23 in one
// fma leaves the rounded integer in the low bits of the sum; the distance of
// v inv from it, again one fma, tells whether any of the eight is close enough
// to a half-integer to be looked at exactly.
__device__ __forceinline__ uint2 i8_codes8(float (&v)[8], const I8RowScale& r) {
    if (r.inv == 0.0f) return make_uint2(0u, 0u);
    if (r.f != 1.0f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r.f;
    }
    constexpr float kMagic = 12582912.0f;
    uint32_t t[8];
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float m = fmaf(v[e], r.inv, kMagic);
        far = fmaxf(far, fabsf(fmaf(v[e], r.inv, kMagic - m)));
        t[e] = __float_as_uint(m);
    }
    if (far > 0.5f - 0x1p-12f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = static_cast<uint32_t>(i8_code_exact(v[e], r.inv, r.a));
    }
    return make_uint2(__byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410));
}

// max(m, |v|) that keeps a NaN.
__device__ __forceinline__ float absmax_nan(float m, float v) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(m), "f"(fabsf(v)));
    return d;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& a, float (&v)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// v times eight channel scales, one rounding to fp32 each (the input gradient
// folds the scales into dY).
__device__ __forceinline__ void i8_scale8(const float* chan, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(chan)), b = __ldg(reinterpret_cast<const float4*>(chan) + 1);
    v[0] = __fmul_rn(v[0], a.x), v[1] = __fmul_rn(v[1], a.y), v[2] = __fmul_rn(v[2], a.z);
    v[3] = __fmul_rn(v[3], a.w), v[4] = __fmul_rn(v[4], b.x), v[5] = __fmul_rn(v[5], b.y);
    v[6] = __fmul_rn(v[6], b.z), v[7] = __fmul_rn(v[7], b.w);
}

// Eight consecutive values of a row as fp32, times the channel scales when given.
template <int SRC, bool SCALED>
__device__ __forceinline__ void i8_load8(const void* row, const float* chan, int64_t j, float (&v)[8]) {
    if (SRC == kSrcF32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + j);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + j));
        if (SRC == kSrcBf16) {
            unpack_bf16x8(a, v);
        } else {
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = f16_bits_to_f32(static_cast<uint16_t>(w[i] & 0xFFFFu));
                v[2 * i + 1] = f16_bits_to_f32(static_cast<uint16_t>(w[i] >> 16));
            }
        }
    }
    if (SCALED) i8_scale8(chan + j, v);
}

// One CTA per row; the row's values stay in registers when it has at most
// 8 * NV * blockDim.x of them (NV > 0), else they are read twice (NV == 0).
// len % 8 == 0.
// BESIDE: the kernel before this one (the adapter's product of the same call)
// started after everything before it was complete and touches nothing of this
// one's, so the two run side by side; waiting for it comes last, so that the
// kernel after this one finds both complete.
template <int SRC, bool SCALED, bool BESIDE, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) i8_quantize_rows_kernel(const void* __restrict__ in, int64_t len,
                                                                   const float* __restrict__ chan,
                                                                   int8_t* __restrict__ codes, int64_t ldc,
                                                                   float* __restrict__ scale) {
    constexpr int ESIZE = SRC == kSrcF32 ? 4 : 2;
    constexpr int KEEP = NV > 0 ? NV : 1;
    __shared__ uint32_t s_max[THREADS / 32];
    if (!BESIDE) griddep_wait();    // everything before this kernel is complete ...
    griddep_launch_dependents();    // ... so the kernel after it may read what came before
    const int64_t row = blockIdx.x;
    const void* src = static_cast<const uint8_t*>(in) + row * len * ESIZE;
    int8_t* dst = codes + row * ldc;
    const int64_t nvec = len / 8;
    float v[KEEP][8];
    float top = 0.0f;
    if (NV > 0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int64_t j = threadIdx.x + static_cast<int64_t>(i) * THREADS;
            if (j < nvec) {
                i8_load8<SRC, SCALED>(src, chan, j * 8, v[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = absmax_nan(top, v[i][e]);
    } else {
        for (int64_t j = threadIdx.x; j < nvec; j += THREADS) {
            i8_load8<SRC, SCALED>(src, chan, j * 8, v[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = absmax_nan(top, v[0][e]);
        }
    }
    // the bits of magnitudes order as the magnitudes do, a NaN above infinity
    uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top) & 0x7FFFFFFFu);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
    __syncthreads();
    mx = __reduce_max_sync(0xFFFFFFFFu, (threadIdx.x & 31) < THREADS / 32 ? s_max[threadIdx.x & 31] : 0u);
    const I8RowScale r = i8_row_scale(mx);
    if (threadIdx.x == 0) scale[row] = r.scale;
    auto put = [&](int64_t j, float (&x)[8]) { *reinterpret_cast<uint2*>(dst + j * 8) = i8_codes8(x, r); };
    if (NV > 0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int64_t j = threadIdx.x + static_cast<int64_t>(i) * THREADS;
            if (j < nvec) put(j, v[i]);
        }
    } else {
        for (int64_t j = threadIdx.x; j < nvec; j += THREADS) {
            i8_load8<SRC, SCALED>(src, chan, j * 8, v[0]);
            put(j, v[0]);
        }
    }
    if (BESIDE) griddep_wait();
}

}  // namespace lbq
