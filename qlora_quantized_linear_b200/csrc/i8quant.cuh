// i8quant.cuh -- symmetric 8-bit quantization of matrix rows: one scale per
// row (per token of an activation, per output channel of a weight).
//
//   amax = max_j |v_j|,  scale = fp32(amax / 127),
//   code_j = 127 v_j / amax rounded to the nearest integer, ties to even.
//
// The codes are those of the exact quotient, so they do not depend on how a
// reciprocal rounds; bf16 data meets exact ties often (v = amax / 2 is 63.5).
// The fast path multiplies by inv = fp32(127 / amax), 2^-24 relative off: for
// |v inv| <= 127 the exact product lies within 2^-17 of the quotient, and the
// rounded value is right unless it lies within 2^-16 of a half-integer.  Those
// elements are compared exactly: in fp32 where the values are short (ties are
// common in bf16), else 127 v with the half-integer times amax in fp64, where
// both products are exact (24 + 8 bits).
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
    float f;      // power of two applied to the values first (rows of very small or large values)
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
        // 127 / amax overflows below 2^-121 and 127 v above 2^121: such rows are
        // brought near 1 first (exact for every value that has a code but 0)
        r.f = a < 0x1p-60f ? 0x1p100f : a > 0x1p60f ? 0x1p-100f : 1.0f;
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

// Two fp32 values in a register pair and Blackwell's packed operations on them
// (each half rounds as the scalar operation does).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// max(m, |a|, |b|), a NaN kept.
__device__ __forceinline__ float absmax3(float m, float a, float b) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
    return d;
}

// The codes of eight values, first in the low byte.  v inv + 1.5 * 2^23 in one
// fma leaves the rounded integer in the low bits of the sum; the distance of
// v inv from it, again one fma, tells whether any of the eight is close enough
// to a half-integer to be looked at exactly.  SHORT: the values have at most
// 11 significant bits (bf16, fp16); there exact ties are common, and
// e = 127 v - q a is exact in one fma (both products have at most 18 bits, and
// near a half-integer v is at least a / 254), so that 2 |e| against a decides.
template <bool SHORT>
__device__ __forceinline__ uint2 i8_codes8(f32x2 (&v)[4], const I8RowScale& r) {
    if (r.inv == 0.0f) return make_uint2(0u, 0u);
    if (r.f != 1.0f) {
        const f32x2 f = pack2(r.f, r.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], f);
    }
    constexpr float kMagic = 12582912.0f;
    const f32x2 inv = pack2(r.inv, r.inv), magic = pack2(kMagic, kMagic), minus = pack2(-1.0f, -1.0f);
    float t[8];
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f32x2 m = fma2(v[e], inv, magic);
        const float2 d = unpack2(fma2(v[e], inv, fma2(m, minus, magic))), q = unpack2(m);
        far = absmax3(far, d.x, d.y);
        t[2 * e] = q.x;
        t[2 * e + 1] = q.y;
    }
    if (far > 0.5f - 0x1p-16f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 vv = unpack2(v[e >> 1]);
            const float ve = e & 1 ? vv.y : vv.x;
            if (SHORT) {
                const float q = t[e] - kMagic;
                const float d = fmaf(-q, r.a, 127.0f * ve);
                const float over = 2.0f * fabsf(d) - r.a;
                const bool odd = (__float_as_uint(t[e]) & 1u) != 0;
                if (over > 0.0f || (over == 0.0f && odd)) t[e] += copysignf(1.0f, d);
            } else {
                t[e] = __uint_as_float(static_cast<uint32_t>(i8_code_exact(ve, r.inv, r.a)));
            }
        }
    }
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(t[e]);
    return make_uint2(__byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410));
}

__device__ __forceinline__ float absmax8(float m, const f32x2 (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 x = unpack2(v[e]);
        m = absmax3(m, x.x, x.y);
    }
    return m;
}

// v times eight channel scales, one rounding to fp32 each (the input gradient
// folds the scales into dY).
__device__ __forceinline__ void i8_scale8(const float* chan, f32x2 (&v)[4]) {
    const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(chan));
    const ulonglong2 b = __ldg(reinterpret_cast<const ulonglong2*>(chan) + 1);
    v[0] = mul2(v[0], a.x), v[1] = mul2(v[1], a.y), v[2] = mul2(v[2], b.x), v[3] = mul2(v[3], b.y);
}

// Eight consecutive values of a row as they are stored.
template <int SRC>
struct I8Raw {
    uint4 lo, hi;          // hi: fp32 only
    __device__ __forceinline__ void zero() { lo = hi = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const void* row, int64_t j) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + j * (SRC == kSrcF32 ? 4 : 2));
        lo = __ldg(p);
        if (SRC == kSrcF32) hi = __ldg(p + 1);
    }
    __device__ __forceinline__ void values(f32x2 (&v)[4]) const {
        const uint32_t w[4] = {lo.x, lo.y, lo.z, lo.w};
        if (SRC == kSrcF32) {
            v[0] = pack2(__uint_as_float(lo.x), __uint_as_float(lo.y));
            v[1] = pack2(__uint_as_float(lo.z), __uint_as_float(lo.w));
            v[2] = pack2(__uint_as_float(hi.x), __uint_as_float(hi.y));
            v[3] = pack2(__uint_as_float(hi.z), __uint_as_float(hi.w));
        } else if (SRC == kSrcBf16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = pack2(f16_bits_to_f32(static_cast<uint16_t>(w[i] & 0xFFFFu)),
                             f16_bits_to_f32(static_cast<uint16_t>(w[i] >> 16)));
        }
    }
};

// Few rows: one CTA per row, which stays in registers as it was stored (NV > 0:
// at most 8 NV blockDim.x values) between its maximum and its codes, or is read
// twice (NV == 0).  len % 8 == 0.
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
    constexpr bool SHORT = SRC != kSrcF32 && !SCALED;
    __shared__ uint32_t s_max[THREADS / 32];
    if (!BESIDE) griddep_wait();    // everything before this kernel is complete ...
    griddep_launch_dependents();    // ... so the kernel after it may read what came before
    const int64_t nvec = len / 8, row = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const void* src = static_cast<const uint8_t*>(in) + row * len * ESIZE;
    int8_t* dst = codes + row * ldc;
    I8Raw<SRC> raw[KEEP];
    auto value8 = [&](const I8Raw<SRC>& x, int64_t j, f32x2 (&v)[4]) {
        x.values(v);
        if (SCALED) i8_scale8(chan + j * 8, v);
    };
    float top = 0.0f;
    if (NV > 0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int64_t j = threadIdx.x + static_cast<int64_t>(i) * THREADS;
            if (j < nvec) raw[i].load(src, j * 8);
            else raw[i].zero();
        }
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int64_t j = threadIdx.x + static_cast<int64_t>(i) * THREADS;
            if (j < nvec) {
                f32x2 v[4];
                value8(raw[i], j, v);
                top = absmax8(top, v);
            }
        }
    } else {
        for (int64_t j = threadIdx.x; j < nvec; j += THREADS) {
            f32x2 v[4];
            raw[0].load(src, j * 8);
            value8(raw[0], j, v);
            top = absmax8(top, v);
        }
    }
    // the bits of magnitudes order as the magnitudes do, a NaN above infinity
    uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top) & 0x7FFFFFFFu);
    if (lane == 0) s_max[threadIdx.x >> 5] = mx;
    __syncthreads();
    mx = __reduce_max_sync(0xFFFFFFFFu, lane < THREADS / 32 ? s_max[lane] : 0u);
    const I8RowScale r = i8_row_scale(mx);
    if (threadIdx.x == 0) scale[row] = r.scale;
    if (NV > 0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int64_t j = threadIdx.x + static_cast<int64_t>(i) * THREADS;
            if (j < nvec) {
                f32x2 v[4];
                value8(raw[i], j, v);
                *reinterpret_cast<uint2*>(dst + j * 8) = i8_codes8<SHORT>(v, r);
            }
        }
    } else {
        for (int64_t j = threadIdx.x; j < nvec; j += THREADS) {
            f32x2 v[4];
            raw[0].load(src, j * 8);
            value8(raw[0], j, v);
            *reinterpret_cast<uint2*>(dst + j * 8) = i8_codes8<SHORT>(v, r);
        }
    }
    if (BESIDE) griddep_wait();
}

}  // namespace lbq
