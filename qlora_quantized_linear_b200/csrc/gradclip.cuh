// gradclip.cuh -- the Euclidean norm of many tensors together, and the tensors
// scaled so that it is at most max_norm:
//
//   total = sum over all tensors and elements g^2          (fp64)
//   norm  = sqrt(total),  coef = fp32(min(1, max_norm / (norm + 1e-6)))
//   out   = g * coef in fp32, rounded to the tensor's type
//
// HBM-bound: every gradient is read once for the norm and once more for the
// scaling.  One persistent CTA per SM takes an equal, contiguous range of the
// 2 KB chunks of all tensors.  The tensors come as kernel arguments; a CTA
// copies the few that its range meets to shared memory first (walking the
// arguments where they are costs a constant-cache miss per step: 9 us of a
// small call).  A warp takes every 16th chunk of its CTA's range and feeds
// itself by bulk copies through a ring of its own, so that the loads never wait
// for the sums (192 KB in flight per SM).  Between the two phases the CTAs meet
// at a grid barrier (a cooperative launch); what the rings hold by then is
// scaled without another read, and the rest is read again from the last chunk
// backwards, the latest of it from L2.
//
// Measured: 42 M fp32 values in 448 tensors in 85 us.  Each value read and
// written once is 51 us at the copy rate; the second read of what neither the
// rings nor L2 held (105 MB of 168) makes it 67 us, and the ramps of the two
// phases and the barrier between them the rest.  168 M bf16 values in 448
// tensors: 172 us, 103 us at one read and one write.
//
// The squares of a lane's four 16-byte pieces of a chunk are added in fp32, in
// chains of four and then in pairs (at most 7 roundings), when the sum is in a
// safe range, else in fp64; all else is added in fp64.  Every sum has a fixed
// order (lanes, warps, CTAs), so the norm does not depend on scheduling.
#pragma once

#include "common.cuh"

namespace lbq {

enum GradType : int { kGradF32 = LBQ_F32, kGradBf16 = LBQ_BF16, kGradF16 = LBQ_F16 };

constexpr int kClipThreads = 512;
constexpr int kClipWarps = kClipThreads / 32;
constexpr int kClipVecs = 4;                          // 16-byte pieces per lane and chunk
constexpr int kClipChunk = kClipVecs * 32 * 16;       // 2 KB
constexpr int kClipSlots = 6;                         // chunks of a warp's ring
constexpr int kClipRing = kClipWarps * kClipSlots * kClipChunk;
constexpr uint32_t kClipL2 = 80u << 20;               // bytes of a launch that L2 is asked to hold between the phases
constexpr int kClipMaxCtas = 256;                     // CTAs of a launch
constexpr int kClipTable = 976;                       // tensors per launch (kernel arguments are below 32764 bytes)

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
    uint32_t chunks;                     // of this launch
    uint16_t first[kClipMaxCtas + 2];    // the tensor of each CTA's first chunk, then the last tensor
    alignas(16) ClipEntry e[CAP];
};

// Shared memory of a CTA: the rings, then the tensors of its range.
template <int CAP>
constexpr int clip_smem_bytes() {
    return kClipRing + CAP * static_cast<int>(sizeof(ClipEntry));
}

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

template <int TYPE>
__device__ __forceinline__ float grad_f32(uint32_t w, int hi) {
    if (TYPE == kGradF32) return __uint_as_float(w);
    const uint32_t h = hi ? w >> 16 : w & 0xFFFFu;
    return TYPE == kGradBf16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(static_cast<uint16_t>(h));
}

// Sum of the squares of a 16-byte piece in fp32: chains of four.
template <int TYPE>
__device__ __forceinline__ float grad_sumsq32(const uint4& r) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = grad_f32<TYPE>(w[i], 0);
        s = fmaf(a, a, s);
    }
    if (TYPE != kGradF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float b = grad_f32<TYPE>(w[i], 1);
            t = fmaf(b, b, t);
        }
    }
    return s + t;
}

template <int TYPE>
__device__ __forceinline__ double grad_sumsq64(const uint4& r) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double a = grad_f32<TYPE>(w[i], 0);
        d = fma(a, a, d);
        if (TYPE != kGradF32) {
            const double b = grad_f32<TYPE>(w[i], 1);
            d = fma(b, b, d);
        }
    }
    return d;
}

// The same of four pieces in fp64; out of line, so that no part of it runs
// where it is not needed.
template <int TYPE>
__device__ __noinline__ double grad_sumsq_far(uint4 a, uint4 b, uint4 c, uint4 d) {
    return (grad_sumsq64<TYPE>(a) + grad_sumsq64<TYPE>(b)) + (grad_sumsq64<TYPE>(c) + grad_sumsq64<TYPE>(d));
}

// Of a lane's four pieces.  In fp32 it is safe when it lies in [2^-66, 2^100]:
// no square overflowed and what squares below the normal range lost is under
// 2^-50 of it.
template <int TYPE>
__device__ __forceinline__ double grad_sumsq(const uint4 (&r)[4]) {
    const float s = (grad_sumsq32<TYPE>(r[0]) + grad_sumsq32<TYPE>(r[1])) +
                    (grad_sumsq32<TYPE>(r[2]) + grad_sumsq32<TYPE>(r[3]));
    double d = static_cast<double>(s);
    if (!(s >= 0x1p-66f && s <= 0x1p100f)) {
        uint32_t any = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= r[i].x | r[i].y | r[i].z | r[i].w;
        d = 0.0;
        if (any != 0u) d = grad_sumsq_far<TYPE>(r[0], r[1], r[2], r[3]);
    }
    return d;
}

template <int TYPE>
__device__ __forceinline__ uint32_t grad_scale_word(uint32_t w, float c) {
    if (TYPE == kGradF32) return __float_as_uint(__fmul_rn(__uint_as_float(w), c));
    const float a = __fmul_rn(grad_f32<TYPE>(w, 0), c), b = __fmul_rn(grad_f32<TYPE>(w, 1), c);
    if (TYPE == kGradBf16) return pack_bf16x2_rn(a, b);
    return static_cast<uint32_t>(f32_to_f16_bits(a)) | (static_cast<uint32_t>(f32_to_f16_bits(b)) << 16);
}

// By the tensor's type, once per chunk.
__device__ __forceinline__ double grad_sumsq_of(const uint4 (&r)[4], int type) {
    if (type == kGradF32) return grad_sumsq<kGradF32>(r);
    return type == kGradBf16 ? grad_sumsq<kGradBf16>(r) : grad_sumsq<kGradF16>(r);
}

template <int TYPE>
__device__ __forceinline__ void grad_scale(uint4 (&r)[4], float c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i].x = grad_scale_word<TYPE>(r[i].x, c);
        r[i].y = grad_scale_word<TYPE>(r[i].y, c);
        r[i].z = grad_scale_word<TYPE>(r[i].z, c);
        r[i].w = grad_scale_word<TYPE>(r[i].w, c);
    }
}

__device__ __forceinline__ void grad_scale_of(uint4 (&r)[4], int type, float c) {
    if (type == kGradF32) grad_scale<kGradF32>(r, c);
    else if (type == kGradBf16) grad_scale<kGradBf16>(r, c);
    else grad_scale<kGradF16>(r, c);
}

// L2 eviction policies: the gradients of the last kClipL2 bytes stay as long as
// they can, the other gradients and the outputs make room first.  The scaling's
// own reads keep the first read's policy, although nothing reads them a third
// time: with evict_first there 20 M fp32 values took 62 us instead of 57 and 168 M
// bf16 values 200 instead of 197, and what runs next was no faster for it (five
// passes over another 96 MB: 85 us after either, 88 with an empty L2; a read of
// the outputs: 45 us after 42 M values, 24.5 after 20 M).
__device__ __forceinline__ uint64_t l2_policy(bool last) {
    uint64_t p;
    if (last) asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    else asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void bulk_load_hint(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
        ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(pol) : "memory");
}

// A generic load, also of kernel arguments (which a thread's own index would
// otherwise read through the constant cache one address at a time).
__device__ __forceinline__ uint4 ld_generic(const void* p) {
    uint4 r;
    asm volatile("ld.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}

__device__ __forceinline__ void st_hint(void* a, const uint4& r, uint64_t pol) {
    asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;"
                 ::"l"(a), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "l"(pol) : "memory");
}

// The first or last piece of a tensor that does not fill 16 bytes: elements
// outside [lead, end) read as zero.
__device__ __forceinline__ uint4 grad_load_part(const ClipEntry& e, int64_t at) {
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

// A piece whose output is not 16-byte aligned or that the tensor does not fill.
__device__ __forceinline__ void grad_store_part(const ClipEntry& e, int64_t at, const uint4& r) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if (e.type == kGradF32) {
        uint32_t* o = reinterpret_cast<uint32_t*>(e.out) + at;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + i >= e.lead && at + i < e.end) o[i] = w[i];
    } else {
        uint16_t* o = reinterpret_cast<uint16_t*>(e.out) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + i >= e.lead && at + i < e.end) o[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
}

// A chunk of whole pieces to an output that starts d bytes past a 16-byte
// boundary: every lane joins the last d bytes of the piece before its own (its
// neighbour's, or the last lane's previous one) with the first 16 - d of its
// own and stores 16 aligned bytes.  The chunk's first 16 - d and last d bytes
// go out in halfwords.  `o` is the lane's first piece.
__device__ __forceinline__ void grad_store_shifted(uint8_t* o, const uint4 (&v)[kClipVecs], int d, int lane, uint64_t pol) {
    const int s = 16 - d, wo = s >> 2, bits = (s & 3) * 8;
#pragma unroll
    for (int i = 0; i < kClipVecs; ++i) {
        const uint4 give = (lane == 31 && i > 0) ? v[i > 0 ? i - 1 : 0] : v[i];
        uint32_t w[9];
        w[0] = __shfl_sync(0xFFFFFFFFu, give.x, (lane + 31) & 31);
        w[1] = __shfl_sync(0xFFFFFFFFu, give.y, (lane + 31) & 31);
        w[2] = __shfl_sync(0xFFFFFFFFu, give.z, (lane + 31) & 31);
        w[3] = __shfl_sync(0xFFFFFFFFu, give.w, (lane + 31) & 31);
        w[4] = v[i].x, w[5] = v[i].y, w[6] = v[i].z, w[7] = v[i].w, w[8] = 0u;
        if (wo & 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = w[j + 1];
        }
        if (wo & 2) {
#pragma unroll
            for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
        }
        uint4 r;
        r.x = __funnelshift_r(w[0], w[1], bits);
        r.y = __funnelshift_r(w[1], w[2], bits);
        r.z = __funnelshift_r(w[2], w[3], bits);
        r.w = __funnelshift_r(w[3], w[4], bits);
        if (i > 0 || lane > 0) st_hint(o + i * 512 - d, r, pol);
    }
    if (lane == 0 || lane == 31) {
        const uint4 e = lane == 0 ? v[0] : v[kClipVecs - 1];
        const uint32_t w[4] = {e.x, e.y, e.z, e.w};
        uint16_t* h = reinterpret_cast<uint16_t*>(lane == 0 ? o : o + (kClipVecs - 1) * 512);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (lane == 0 ? 2 * j < s : 2 * j >= s) h[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
}

// A tensor of the range and what the walk over its chunks needs of it, in
// registers: neighbouring chunks mostly belong to the same one.
struct ClipCursor {
    const ClipEntry* ent;
    int fn, ti;
    uint32_t chunk0, next0;     // first chunk of the tensor and of the one after it
    const uint8_t* g;
    uint8_t* out;
    int64_t end;
    int type, lead, log_per;    // 2^log_per elements in 16 bytes
    __device__ __forceinline__ ClipCursor(const ClipEntry* e, int n) : ent(e), fn(n), ti(0) { set(); }
    __device__ __forceinline__ void set() {
        if (fn < 1) return;
        const ClipEntry& e = ent[ti];
        chunk0 = e.chunk0;
        next0 = ti + 1 < fn ? ent[ti + 1].chunk0 : 0xFFFFFFFFu;
        g = e.g;
        out = e.out;
        end = e.end;
        type = e.type;
        lead = e.lead;
        log_per = type == kGradF32 ? 2 : 3;
    }
    __device__ __forceinline__ void seek(uint32_t c) {
        while (c >= next0) ++ti, set();
        while (c < chunk0) --ti, set();
    }
};

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
    __shared__ uint64_t s_full[kClipWarps][kClipSlots];
    __shared__ double s_sum[kClipWarps];
    __shared__ int s_last, s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this CTA's chunks cb .. cb + cn - 1; the warp's are cb + warp + 16 q, q < nq
    const uint32_t cb = static_cast<uint32_t>(static_cast<uint64_t>(tab.chunks) * blockIdx.x / gridDim.x);
    const int cn = static_cast<int>(static_cast<uint64_t>(tab.chunks) * (blockIdx.x + 1) / gridDim.x - cb);
    const int nq = cn > warp ? (cn - 1 - warp) / kClipWarps + 1 : 0;
    uint8_t* ring = clip_smem + warp * kClipSlots * kClipChunk;
    uint64_t* full = s_full[warp];
    if (lane == 0) {
        for (int i = 0; i < kClipSlots; ++i) mbar_init(&full[i], 1);
        if (warp == 0) s_abort = 0;
        fence_mbar_init();
    }
    // the tensors of this range, from the arguments to shared memory by all threads at once
    ClipEntry* ent = reinterpret_cast<ClipEntry*>(clip_smem + kClipRing);
    const int f0 = tab.first[blockIdx.x], fn = tab.count > 0 ? tab.first[blockIdx.x + 1] - f0 + 1 : 0;
    bool same = true;
#pragma unroll
    for (int i0 = 0; i0 < CAP; i0 += kClipThreads) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        if (i < fn) {
            const uint4* src = reinterpret_cast<const uint4*>(tab.e + f0 + i);
            uint4* dst = reinterpret_cast<uint4*>(ent + i);
            const uint4 p = ld_generic(src);                    // g, out
            same &= p.x == p.z && p.y == p.w;
            dst[0] = p;
            dst[1] = ld_generic(src + 1);
        }
    }
    const bool inplace = __syncthreads_and(same);           // of the whole range
    const uint64_t drop = l2_policy(false), hold = l2_policy(true);
    const int held = cn - static_cast<int>(kClipL2 / kClipChunk / gridDim.x);      // first chunk to hold in L2
    // the whole pieces of chunk q to its slot; piece p of a tensor holds the
    // elements p << log_per and on
    ClipCursor tl(ent, fn), tc(ent, fn);    // tensors of the chunk last loaded and of the one worked on
    auto load = [&](int q) {
        tl.seek(cb + warp + q * kClipWarps);
        if (lane == 0) {
            const int lp = tl.log_per;
            const int64_t p0 = static_cast<int64_t>(cb + warp + q * kClipWarps - tl.chunk0) * (kClipChunk / 16);
            const int64_t lo = max(p0, static_cast<int64_t>(tl.lead > 0));
            const int64_t hi = min(p0 + kClipChunk / 16, tl.end >> lp);
            const uint32_t bytes = hi > lo ? static_cast<uint32_t>(hi - lo) * 16 : 0;
            uint64_t* bar = &full[q % kClipSlots];
            mbar_arrive_expect_tx(bar, bytes);
            if (bytes)
                bulk_load_hint(ring + (q % kClipSlots) * kClipChunk + (lo - p0) * 16, tl.g + lo * 16, bytes, bar,
                               MODE == kClipFused && warp + q * kClipWarps >= held ? hold : drop);
        }
    };
    uint32_t phase = 0;                     // a bit per slot
    auto wait = [&](int q) {
        const int slot = q % kClipSlots;
        mbar_wait(&full[slot], (phase >> slot) & 1u, &s_abort);
        phase ^= 1u << slot;
    };
    // the lane's pieces of chunk q, which begin at element `at` and every 32 pieces on; true when all are whole
    auto pieces = [&](int q, int64_t at, uint4 (&r)[kClipVecs]) {
        const uint4* slot = reinterpret_cast<const uint4*>(ring + (q % kClipSlots) * kClipChunk) + lane;
#pragma unroll
        for (int i = 0; i < kClipVecs; ++i) r[i] = slot[i * 32];
        const int64_t first = at - (static_cast<int64_t>(lane) << tc.log_per);
        if (first >= tc.lead && first + ((kClipChunk / 16) << tc.log_per) <= tc.end) return true;
        const int per = 1 << tc.log_per;
#pragma unroll
        for (int i = 0; i < kClipVecs; ++i) {
            const int64_t a = at + (i * 32 << tc.log_per);
            if (a < tc.lead || a + per > tc.end)
                r[i] = a < tc.end ? grad_load_part(ent[tc.ti], a) : make_uint4(0u, 0u, 0u, 0u);
        }
        return false;
    };
    if (MODE != kClipScale) {
        double acc = 0.0;
        for (int q = 0; q < nq && q < kClipSlots; ++q) load(q);
        for (int q = 0; q < nq; ++q) {
            const uint32_t c = cb + warp + q * kClipWarps;
            tc.seek(c);
            const int64_t at = static_cast<int64_t>((c - tc.chunk0) * uint64_t(kClipChunk / 16) + lane) << tc.log_per;
            wait(q);
            uint4 r[kClipVecs];
            pieces(q, at, r);
            __syncwarp();                                       // the slot is read
            if (q + kClipSlots < nq) load(q + kClipSlots);
            acc += grad_sumsq_of(r, tc.type);
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
    if (coef == 1.0f && inplace) return;                    // nothing to change, and no load is in flight
    if (MODE == kClipScale)
        for (int q = nq - 1; q >= 0 && q >= nq - kClipSlots; --q) load(q);
    for (int q = nq - 1; q >= 0; --q) {
        const uint32_t c = cb + warp + q * kClipWarps;
        tc.seek(c);
        const int64_t at = static_cast<int64_t>((c - tc.chunk0) * uint64_t(kClipChunk / 16) + lane) << tc.log_per;
        if (MODE == kClipScale || q < nq - kClipSlots) wait(q);
        uint4 r[kClipVecs];
        const bool whole = pieces(q, at, r);
        __syncwarp();                                           // the slot is read
        if (q >= kClipSlots) load(q - kClipSlots);
        if (coef == 1.0f && tc.g == tc.out) continue;           // this tensor is in place
        uint8_t* o = tc.out + (at << (4 - tc.log_per));
        const int d = static_cast<int>(reinterpret_cast<uintptr_t>(tc.out) & 15u);
        grad_scale_of(r, tc.type, coef);
        if (!whole) {
#pragma unroll
            for (int i = 0; i < kClipVecs; ++i) grad_store_part(ent[tc.ti], at + (i * 32 << tc.log_per), r[i]);
        } else if (d == 0) {
#pragma unroll
            for (int i = 0; i < kClipVecs; ++i) st_hint(o + i * 512, r[i], drop);
        } else {
            grad_store_shifted(o, r, d, lane, drop);
        }
    }
}

}  // namespace lbq
