// gradclip.cuh -- the Euclidean norm of many tensors together, and the tensors
// scaled so that it is at most max_norm:
//
//   total = sum over all tensors and elements g^2          (fp64)
//   norm  = sqrt(total),  coef = fp32(min(1, max_norm / (norm + 1e-6)))
//   out   = g * coef in fp32, rounded to the tensor's type
//
// HBM-bound: every gradient is read once for the norm and once more for the
// scaling.  One persistent CTA per SM walks over 4 KB chunks of all tensors
// (a warp per chunk), so a launch costs the same for 14 tensors as for 448.
// Between the two phases the CTAs meet at a grid barrier (a cooperative
// launch); each warp keeps its first chunks in shared memory meanwhile, and
// reads the others again from the last backwards, when the L2 cache still
// holds the latest of them.
//
// The squares of a 16-byte piece are added in fp32 when the sum is in a safe
// range, else in fp64; the pieces are added in fp64.  Every sum has a fixed
// order (lanes, warps, CTAs), so the norm does not depend on scheduling.
#pragma once

#include "common.cuh"

namespace lbq {

enum GradType : int { kGradF32 = LBQ_F32, kGradBf16 = LBQ_BF16, kGradF16 = LBQ_F16 };

constexpr int kClipThreads = 512;
constexpr int kClipWarps = kClipThreads / 32;
constexpr int kClipVecs = 8;                          // 16-byte pieces per lane and chunk
constexpr int kClipChunk = kClipVecs * 32 * 16;       // 4 KB
constexpr int kClipKeep = 3;                          // chunks a warp keeps in shared memory
constexpr int kClipSmem = kClipWarps * kClipKeep * kClipChunk;
constexpr int kClipMaxCtas = 1024;                    // partial sums in the workspace, per launch
constexpr int kClipTable = 1000;                      // tensors per launch (kernel arguments are below 32764 bytes)

struct ClipEntry {
    const uint8_t* g;      // rounded down to 16 bytes
    uint8_t* out;          // of the same element: out - lead * size
    int64_t end;           // lead + numel, in elements
    uint32_t chunk0;       // chunks of the tensors before it
    uint16_t type;
    uint16_t lead;         // elements between g and the tensor's first one
};

template <int CAP>
struct ClipTable {
    int count;
    uint32_t chunks;                // of this launch
    ClipEntry e[CAP];
};

struct ClipWork {
    uint32_t* bar;                  // {arrivals, generation}: arrivals 0 between calls
    double* part;                   // [nparts] partial sums, one per CTA and launch
    double* total;                  // the sum, for the launches that only scale
    float* norm;                    // output
    float max_norm;
    int part0;                      // first partial sum of this launch
    int nparts;                     // of all launches
};

enum ClipMode : int { kClipSum = 0, kClipSumLast = 1, kClipScale = 2, kClipFused = 3 };

__device__ __forceinline__ float grad_f32(uint32_t w, int type, int hi) {
    if (type == kGradF32) return __uint_as_float(w);
    const uint32_t h = hi ? w >> 16 : w & 0xFFFFu;
    return type == kGradBf16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(static_cast<uint16_t>(h));
}

// Sum of the squares of a 16-byte piece.  In fp32 it is safe when it lies in
// [2^-66, 2^100]: no square overflowed and what squares below the normal
// range lost is under 2^-60 of it.
__device__ __forceinline__ double grad_sumsq(const uint4& r, int type) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    float s = 0.0f;
    if (type == kGradF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fmaf(__uint_as_float(w[i]), __uint_as_float(w[i]), s);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = grad_f32(w[i], type, 0), b = grad_f32(w[i], type, 1);
            s = fmaf(a, a, s);
            s = fmaf(b, b, s);
        }
    }
    if (s >= 0x1p-66f && s <= 0x1p100f) return static_cast<double>(s);
    if ((r.x | r.y | r.z | r.w) == 0u) return 0.0;
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double a = grad_f32(w[i], type, 0);
        d = fma(a, a, d);
        if (type != kGradF32) {
            const double b = grad_f32(w[i], type, 1);
            d = fma(b, b, d);
        }
    }
    return d;
}

__device__ __forceinline__ uint32_t grad_scale_word(uint32_t w, int type, float c) {
    if (type == kGradF32) return __float_as_uint(__fmul_rn(__uint_as_float(w), c));
    const float a = __fmul_rn(grad_f32(w, type, 0), c), b = __fmul_rn(grad_f32(w, type, 1), c);
    if (type == kGradBf16) return pack_bf16x2_rn(a, b);
    return static_cast<uint32_t>(f32_to_f16_bits(a)) | (static_cast<uint32_t>(f32_to_f16_bits(b)) << 16);
}

// The piece at elements [at, at + 16 / size) of a tensor; elements outside
// [lead, end) read as zero.
__device__ __forceinline__ uint4 grad_load(const ClipEntry& e, int64_t at) {
    const int per = e.type == kGradF32 ? 4 : 8;
    if (at >= e.lead && at + per <= e.end) return __ldcg(reinterpret_cast<const uint4*>(e.g + at * (16 / per)));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (e.type == kGradF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + i >= e.lead && at + i < e.end) w[i] = __ldcg(reinterpret_cast<const uint32_t*>(e.g) + at + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + i >= e.lead && at + i < e.end)
                w[i >> 1] |= static_cast<uint32_t>(__ldcg(reinterpret_cast<const uint16_t*>(e.g) + at + i)) << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void grad_store(const ClipEntry& e, int64_t at, const uint4& r) {
    const int per = e.type == kGradF32 ? 4 : 8;
    uint8_t* o = e.out + at * (16 / per);
    if (at >= e.lead && at + per <= e.end && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
        __stcs(reinterpret_cast<uint4*>(o), r);
        return;
    }
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if (e.type == kGradF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + i >= e.lead && at + i < e.end) reinterpret_cast<uint32_t*>(o)[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + i >= e.lead && at + i < e.end)
                reinterpret_cast<uint16_t*>(o)[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
}

// Sum of one value per thread of the CTA, in a fixed order; valid in all threads.
__device__ __forceinline__ double cta_sum(double v, double* s_sum) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kClipWarps; ++w) t += s_sum[w];
    __syncthreads();
    return t;
}

__device__ __forceinline__ double sum_parts(const double* part, int nparts, double* s_sum) {
    double v = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kClipThreads) v += __ldcg(part + i);
    return cta_sum(v, s_sum);
}

template <int MODE, int CAP>
__global__ void __launch_bounds__(kClipThreads, 1)
    grad_clip_kernel(const __grid_constant__ ClipTable<CAP> tab, const __grid_constant__ ClipWork wk) {
    extern __shared__ __align__(128) uint8_t clip_smem[];
    __shared__ double s_sum[kClipWarps];
    __shared__ int s_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t nwarps = gridDim.x * kClipWarps;
    // consecutive chunks go to different SMs
    const uint32_t c0 = warp * gridDim.x + blockIdx.x;
    uint4* keep = reinterpret_cast<uint4*>(clip_smem) + warp * kClipKeep * (kClipChunk / 16) + lane;
    int ti = 0;
    uint32_t done = 0;                      // chunks this warp has taken
    griddep_wait();
    if (MODE != kClipScale) {
        double acc = 0.0;
        for (uint32_t c = c0; c < tab.chunks; c += nwarps, ++done) {
            while (ti + 1 < tab.count && tab.e[ti + 1].chunk0 <= c) ++ti;
            const ClipEntry& e = tab.e[ti];
            const int type = e.type, per = type == kGradF32 ? 4 : 8;
            const int64_t at = (static_cast<int64_t>(c - e.chunk0) * (kClipChunk / 16) + lane) * per;
            uint4 r[kClipVecs];
#pragma unroll
            for (int i = 0; i < kClipVecs; ++i) {
                r[i] = make_uint4(0u, 0u, 0u, 0u);
                if (at + i * 32 * per < e.end) r[i] = grad_load(e, at + i * 32 * per);
            }
#pragma unroll
            for (int i = 0; i < kClipVecs; ++i) acc += grad_sumsq(r[i], type);
            if (MODE == kClipFused && done < kClipKeep) {
#pragma unroll
                for (int i = 0; i < kClipVecs; ++i) keep[done * (kClipChunk / 16) + i * 32] = r[i];
            }
        }
        const double mine = cta_sum(acc, s_sum);
        if (threadIdx.x == 0) {
            wk.part[wk.part0 + blockIdx.x] = mine;
            if (MODE != kClipSum) {
                uint32_t gen;
                asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(gen) : "l"(wk.bar + 1) : "memory");
                __threadfence();
                const bool last = atomicInc(wk.bar, gridDim.x - 1) == gridDim.x - 1;     // back to 0 by the last one
                __threadfence();
                s_last = last;
                if (MODE == kClipFused) {
                    if (last) {
                        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(wk.bar + 1) : "memory");
                    } else {
                        const uint64_t t0 = globaltimer_ns();
                        while (flag_load_acquire(wk.bar + 1) == gen) {
                            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                                record_status(kStatusTimeout);
                                break;
                            }
                        }
                    }
                }
            }
        }
        __syncthreads();
    }
    if (MODE == kClipSum || (MODE == kClipSumLast && !s_last)) return;
    const double total = MODE == kClipScale ? __ldcg(wk.total) : sum_parts(wk.part, wk.nparts, s_sum);
    const double norm = sqrt(total);
    if (MODE != kClipScale && (MODE == kClipSumLast || blockIdx.x == 0) && threadIdx.x == 0) {
        *wk.norm = static_cast<float>(norm);
        *wk.total = total;
    }
    if (MODE == kClipSumLast) return;
    // min(1, x) that keeps a NaN
    const double ratio = static_cast<double>(wk.max_norm) / (norm + 1e-6);
    const float coef = ratio > 1.0 ? 1.0f : static_cast<float>(ratio);
    if (MODE == kClipScale) {
        for (uint32_t c = c0; c < tab.chunks; c += nwarps) ++done;
        ti = tab.count - 1;
    }
    while (done > 0) {
        --done;
        const uint32_t c = c0 + done * nwarps;
        while (tab.e[ti].chunk0 > c) --ti;
        const ClipEntry& e = tab.e[ti];
        if (coef == 1.0f && e.g == e.out) continue;                    // in place and nothing to change
        const int type = e.type, per = type == kGradF32 ? 4 : 8;
        const int64_t at = (static_cast<int64_t>(c - e.chunk0) * (kClipChunk / 16) + lane) * per;
        uint4 r[kClipVecs];
#pragma unroll
        for (int i = 0; i < kClipVecs; ++i) {
            r[i] = make_uint4(0u, 0u, 0u, 0u);
            if (at + i * 32 * per < e.end) {
                if (MODE == kClipFused && done < kClipKeep) r[i] = keep[done * (kClipChunk / 16) + i * 32];
                else r[i] = grad_load(e, at + i * 32 * per);
            }
        }
#pragma unroll
        for (int i = 0; i < kClipVecs; ++i) {
            if (at + i * 32 * per >= e.end) continue;
            uint4 o;
            o.x = grad_scale_word(r[i].x, type, coef);
            o.y = grad_scale_word(r[i].y, type, coef);
            o.z = grad_scale_word(r[i].z, type, coef);
            o.w = grad_scale_word(r[i].w, type, coef);
            grad_store(e, at + i * 32 * per, o);
        }
    }
}

}  // namespace lbq
