// i8quant.cuh -- symmetric 8-bit quantization of matrix rows: one scale per
// row (per token of an activation, per output channel of a weight).
//
//   amax = max_j |v_j|,  scale = fp32(amax / 127),
//   code_j = 127 v_j / amax rounded to the nearest integer, ties to even.
//
// The codes are those of the exact quotient, so they do not depend on how a
// reciprocal rounds; bf16 data meets exact ties often (v = amax / 2 is 63.5).
// The codes come from v inv with inv = 127 / amax rounded up, at most 2^-23
// relative above it: for |v inv| <= 127 the exact product lies within 2^-16 of
// the quotient, and its rounding is right unless it lies that close to a
// half-integer.
//   bf16: a quotient of two 8-bit numbers that is no half-integer is farther
//   away than that (2^-16 relative), so only exact ties are left.  They need
//   127 to divide mantissa(amax) (2 k + 1): either the tie is 63.5, which goes
//   up to the even 64 as inv does, or the mantissa is 254 and inv a power of
//   two, so that the product is exact.  Nothing has to be looked at.
//   fp16 has more such mantissas (127 c for c = 9 .. 16), fp32 any quotient:
//   there a value within 2^-15 of a half-integer (one in 2^14) has 127 v
//   compared with the half-integer times amax in fp64, where both products are
//   exact (24 + 8 bits).
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
    float inv;    // 127 / (amax f), rounded up; 0 for a row without codes
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
        r.inv = __fdiv_ru(127.0f, r.a);
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
// fma leaves the rounded integer in the low bits of the sum.  EXACT: the
// distance of v inv from it, again one fma, tells whether any of the eight is
// close enough to a half-integer to be looked at exactly; bf16 values need no
// look.
template <bool EXACT>
__device__ __forceinline__ uint2 i8_codes8(f32x2 (&v)[4], const I8RowScale& r) {
    if (r.inv == 0.0f) return make_uint2(0u, 0u);
    if (r.f != 1.0f) {
        const f32x2 f = pack2(r.f, r.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], f);
    }
    constexpr float kMagic = 12582912.0f;
    const f32x2 inv = pack2(r.inv, r.inv), magic = pack2(kMagic, kMagic), minus = pack2(-1.0f, -1.0f);
    uint32_t t[8];
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f32x2 m = fma2(v[e], inv, magic);
        if (EXACT) {
            const float2 d = unpack2(fma2(v[e], inv, fma2(m, minus, magic)));
            far = absmax3(far, d.x, d.y);
        }
        const float2 q = unpack2(m);
        t[2 * e] = __float_as_uint(q.x);
        t[2 * e + 1] = __float_as_uint(q.y);
    }
    if (EXACT && far > 0.5f - 0x1p-15f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 vv = unpack2(v[e >> 1]);
            t[e] = static_cast<uint32_t>(i8_code_exact(e & 1 ? vv.y : vv.x, r.inv, r.a));
        }
    }
    return make_uint2(__byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410));
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
// folds the scales into dY).  The scales are 16-byte aligned, no more: two loads
// (of the kind that I8Raw::load explains).
__device__ __forceinline__ void i8_scale8(const float* chan, f32x2 (&v)[4]) {
    f32x2 c[4];
    asm volatile("ld.global.v2.b64 {%0, %1}, [%2];" : "=l"(c[0]), "=l"(c[1]) : "l"(chan));
    asm volatile("ld.global.v2.b64 {%0, %1}, [%2];" : "=l"(c[2]), "=l"(c[3]) : "l"(chan + 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], c[e]);
}

// Eight consecutive values of a row as they are stored.
template <int SRC>
struct I8Raw {
    uint4 lo, hi;          // hi: fp32 only
    // Not the read-only path: this kernel may be resident while the one before it
    // still writes what is read here (tokens, channel scales), and that path is
    // for memory that does not change as long as the kernel lives.  L1 is left to
    // the channel scales, which the CTAs of an SM share (4096 x 14336 scaled rows:
    // 44.7 us, 45.4 without the hint).
    static __device__ __forceinline__ uint4 load16(const uint4* p) {
        uint4 r;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
        return r;
    }
    __device__ __forceinline__ void zero() { lo = hi = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const void* row, int64_t j) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + j * (SRC == kSrcF32 ? 4 : 2));
        lo = load16(p);
        if (SRC == kSrcF32) hi = load16(p + 1);
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

// One CTA per row, which stays in registers (NV > 0: at most 8 NV THREADS values;
// as they were stored, or scaled) between its maximum and its codes, or is read
// twice (NV == 0).  Many rows keep 64 to 112 bytes a thread in flight with up to
// 1024 threads per SM (4096 x 14336 bf16: 28 us, 0.96 of the copy rate; with
// channel scales 45 us, bound by reading them and by the exact check, with 64 of
// a thread's bytes spilled at seven pieces); few rows take as many threads as the
// row has pieces.  len % 8 == 0.
// BESIDE: the kernel before this one (the adapter's product of the same call)
// started after everything before it was complete and touches nothing of this
// one's, so the two run side by side; waiting for it comes last, so that the
// kernel after this one finds both complete.
template <int SRC, bool SCALED, bool BESIDE, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) i8_quantize_rows_kernel(const void* __restrict__ in, int64_t len,
                                                                   const float* __restrict__ chan,
                                                                   int8_t* __restrict__ codes, int64_t ldc,
                                                                   float* __restrict__ scale) {
    constexpr int ESIZE = SRC == kSrcF32 ? 4 : 2;
    constexpr int KEEP = NV > 0 ? NV : 1;
    constexpr bool EXACT = SRC != kSrcBf16 || SCALED;
    __shared__ uint32_t s_max[THREADS / 32];
    if (!BESIDE) griddep_wait();    // everything before this kernel is complete ...
    griddep_launch_dependents();    // ... so the kernel after it may read what came before
    const int64_t nvec = len / 8, row = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const void* src = static_cast<const uint8_t*>(in) + row * len * ESIZE;
    int8_t* dst = codes + row * ldc;
    I8Raw<SRC> raw[KEEP];
    f32x2 held[SCALED ? KEEP : 1][4];            // scaled values stay as they are, others as they were stored
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
                if (SCALED) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) held[i][e] = v[e];
                }
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
                if (SCALED) {
                    *reinterpret_cast<uint2*>(dst + j * 8) = i8_codes8<EXACT>(held[SCALED ? i : 0], r);
                } else {
                    f32x2 v[4];
                    value8(raw[i], j, v);
                    *reinterpret_cast<uint2*>(dst + j * 8) = i8_codes8<EXACT>(v, r);
                }
            }
        }
    } else {
        for (int64_t j = threadIdx.x; j < nvec; j += THREADS) {
            f32x2 v[4];
            raw[0].load(src, j * 8);
            value8(raw[0], j, v);
            *reinterpret_cast<uint2*>(dst + j * 8) = i8_codes8<EXACT>(v, r);
        }
    }
    if (BESIDE) griddep_wait();
}

}  // namespace lbq
