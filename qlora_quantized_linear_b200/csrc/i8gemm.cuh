// i8gemm.cuh -- matrix products in 8-bit integers on the 5th-generation tensor
// cores (tcgen05.mma kind::i8, int32 accumulation in tensor memory), with one
// scale per token and one per output channel, and the low-rank adapter's term:
//
//   forward   Y[t, j]  = (sum_k Xq[t, k] Wq[j, k]) sx[t] sw[j] + s sum_u T[t, u] B[j, u]
//   backward  dX[t, j] = (sum_n Vq[t, n] Wq[n, j]) sv[t]       + s sum_u U[t, u] A[u, j]
//
// The sums of 8-bit products are exact in int32 (127^2 times at most 131072
// terms), whatever their order, so every split of the reduction gives the same
// bits.  Both directions read the one stored copy of the codes Wq [n, k]: in
// the forward the weight tile is the MMA's K-major A operand, in the backward
// the same bytes are its MN-major A operand (a channel row holds 128
// consecutive output features).  The output features are the MMA's M (TMEM
// lanes), the tokens its N, so 32 lanes of a warp hold 32 consecutive output
// features of a token and store 128 contiguous bytes.
//
// The adapter's term is added in fp32 from the fp32 T or U (in bf16 it would
// be the least exact part of the output).
#pragma once

#include "common.cuh"

namespace lbq {

constexpr int kI8MaxReduction = 131072;   // 127^2 * 131072 < 2^31

struct I8Params {
    int m, out, red;           // tokens, output features, reduction length
    const float* row_scale;    // [m] token scales (readable up to the next multiple of 16 tokens)
    const float* out_scale;    // [out] channel scales, or NULL (backward)
    int rank;
    float s;
    const float* T;            // [m, rank] fp32: T (forward) or U (backward)
    const uint16_t* P;         // adapter factor of output feature j: P[j * pj + u * pu]
    int64_t pj, pu;
    float* Y;                  // [m, out]
};

// Instruction descriptor of kind::i8: signed A and B, int32 accumulator,
// shape M x N, A MN-major when TRANS.
__host__ __device__ constexpr uint32_t idesc_i8_s32(int M, int N, bool trans_a) {
    return (2u << 4)                                 // D format: s32
           | (1u << 7)                               // A format: s8
           | (1u << 10)                              // B format: s8
           | (trans_a ? 1u << 15 : 0u)
           | (static_cast<uint32_t>(N >> 3) << 17)   // N / 8
           | (static_cast<uint32_t>(M >> 4) << 24);  // M / 16
}

__device__ __forceinline__ void mma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One 128-byte reduction block of a 128-row A tile: a 128-byte-swizzled tile
// of 128 rows x 128 bytes either way.  K-major: a row is an output feature,
// 32 reduction steps further are 32 bytes further.  MN-major: a row is a
// reduction step, 128 output features wide (one swizzle atom, so the leading
// offset is not used); groups of 8 steps are 1024 bytes apart and 32 steps
// further are 4096 bytes further.
template <bool TRANS>
__device__ __forceinline__ uint64_t i8_a_desc(uint32_t tile, int j) {
    return TRANS ? smem_desc_mn_sw128(tile + j * 4096, 1024, 1024)
                 : smem_desc_k_sw128(tile) + static_cast<uint64_t>(2 * j);
}

// Adapter factors of one output feature, zero beyond the rank.
template <int RP>
__device__ __forceinline__ void i8_load_factor(const I8Params& p, int64_t j, bool ok, float (&b)[RP > 0 ? RP : 1]) {
    if (RP > 0) {
#pragma unroll
        for (int u = 0; u < RP; ++u)
            b[u] = (ok && u < p.rank) ? bf16_bits_to_f32(__ldg(p.P + j * p.pj + u * p.pu)) : 0.0f;
    }
}

// sum_u T[t, u] b[u]; `row` is the same for all lanes of the warp.
template <int RP>
__device__ __forceinline__ float i8_factor_dot(const float* row, int rank, const float (&b)[RP > 0 ? RP : 1]) {
    float d = 0.0f;
    if ((rank & 3) == 0) {
#pragma unroll
        for (int u = 0; u < RP; u += 4) {
            if (u < rank) {
                const float4 t = __ldg(reinterpret_cast<const float4*>(row + u));
                d = fmaf(t.x, b[u], d);
                d = fmaf(t.y, b[u + 1], d);
                d = fmaf(t.z, b[u + 2], d);
                d = fmaf(t.w, b[u + 3], d);
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < RP; ++u)
            if (u < rank) d = fmaf(__ldg(row + u), b[u], d);
    }
    return d;
}

// Y of one output feature j for N consecutive tokens from t.
template <int RP, int N>
__device__ __forceinline__ void i8_store(const I8Params& p, int t, int64_t j, const int (&acc)[N], float so,
                                         const float (&b)[RP > 0 ? RP : 1]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (t + i < p.m) {
            float v = static_cast<float>(acc[i]) * __ldg(p.row_scale + t + i) * so;
            if (RP > 0) v = fmaf(p.s, i8_factor_dot<RP>(p.T + static_cast<int64_t>(t + i) * p.rank, p.rank, b), v);
            p.Y[static_cast<int64_t>(t + i) * p.out + j] = v;
        }
    }
}

// ---------------------------------------------------------------------------
// Few tokens: one CTA per 128 output features x NT tokens x part of the
// reduction.  The CTAs of a cluster hold the parts of one tile; each adds up
// its share of the tokens over the cluster's shared memory.
// ---------------------------------------------------------------------------
constexpr int kI8SplitThreads = 192;      // producer warp, MMA warp, four epilogue warps
constexpr int kI8MaxSplit = 8;

template <int NT>
struct I8SplitCfg {
    static constexpr int kStages = NT <= 16 ? 6 : NT <= 32 ? 5 : NT <= 64 ? 4 : 3;   // two CTAs per SM
    static constexpr int kABytes = 128 * 128;
    static constexpr int kBBytes = NT * 128;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr size_t kBar = size_t(kStages) * kStageBytes;
    static constexpr size_t kBytes = kBar + (2 * kStages + 1) * 8 + 16 + 1024;
    static_assert(size_t(NT) * 512 <= kBar, "the partial sums reuse the ring");
};

template <int NT, bool TRANS, int RP>
__global__ void __launch_bounds__(kI8SplitThreads)
    i8_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ I8Params p) {
    using C = I8SplitCfg<NT>;
    constexpr int S = C::kStages;
    constexpr uint32_t kTmemCols = NT < 32 ? 32 : NT;
    constexpr uint32_t kIdesc = idesc_i8_s32(128, NT, TRANS);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBar);
    uint64_t* empty = full + S;
    uint64_t* dfull = empty + S;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(dfull + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nsplit = static_cast<int>(gridDim.z), part = static_cast<int>(blockIdx.z);
    const int j0 = blockIdx.x * 128, t0 = blockIdx.y * NT;
    const int nblk = (p.red + 127) / 128;
    const int b0 = static_cast<int>(static_cast<int64_t>(nblk) * part / nsplit);
    const int nb = static_cast<int>(static_cast<int64_t>(nblk) * (part + 1) / nsplit) - b0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(dfull, 1);
        *s_abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(s_tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == 0) {
        if (lane == 0) {
            auto load_w = [&](int i) {
                uint8_t* a = smem + (i % S) * C::kStageBytes;
                mbar_arrive_expect_tx(&full[i % S], C::kStageBytes);
                if (TRANS) tma_load_2d(a, &tmW, &full[i % S], j0, (b0 + i) * 128);
                else tma_load_2d(a, &tmW, &full[i % S], (b0 + i) * 128, j0);
            };
            // the weight does not depend on the kernel before this one (which
            // starts only after everything before it is complete), the codes
            // of the tokens do
            const int ahead = nb < S ? nb : S;
            for (int i = 0; i < ahead; ++i) load_w(i);
            griddep_wait();
            griddep_launch_dependents();
            int i = 0;
            for (; i < nb; ++i) {
                if (i >= S) {
                    if (!mbar_wait(&empty[i % S], ((i / S) - 1) & 1, s_abort)) break;
                    load_w(i);
                }
                tma_load_2d(smem + (i % S) * C::kStageBytes + C::kABytes, &tmX, &full[i % S], (b0 + i) * 128, t0);
            }
            for (int d = max(0, i - S); d < i; ++d) mbar_wait_drain(&full[d % S], (d / S) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int i = 0; i < nb; ++i) {
                if (!mbar_wait(&full[i % S], (i / S) & 1, s_abort)) break;
                tc_fence_after();
                const uint32_t a = smem_u32(smem + (i % S) * C::kStageBytes);
                const uint64_t bdesc = smem_desc_k_sw128(a + C::kABytes);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_i8_ss(tmem, i8_a_desc<TRANS>(a, j), bdesc + static_cast<uint64_t>(2 * j), kIdesc,
                              (i > 0 || j > 0) ? 1u : 0u);
                mma_commit(&empty[i % S]);
            }
            mma_commit(dfull);
            mbar_wait_drain(dfull, 0);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        griddep_wait();
        const int quarter = warp & 3;
        const int64_t j = j0 + quarter * 32 + lane;
        const bool ok = j < p.out;
        const bool done = mbar_wait(dfull, 0, s_abort);
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        if (nsplit == 1) {
            float b[RP > 0 ? RP : 1];
            i8_load_factor<RP>(p, j, ok, b);
            const float so = (ok && p.out_scale) ? __ldg(p.out_scale + j) : 1.0f;
#pragma unroll 1
            for (int c = 0; done && c < NT && t0 + c < p.m; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c, r);
                tmem_ld_wait();
                int acc[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = static_cast<int>(r[i]);
                if (ok) i8_store<RP, 16>(p, t0 + c, j, acc, so, b);
            }
        } else if (done) {
            // this part's sums to shared memory: [token][feature]
            int* buf = reinterpret_cast<int*>(smem);
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) buf[(c + i) * 128 + quarter * 32 + lane] = static_cast<int>(r[i]);
            }
        }
    }
    tc_fence_before();
    if (nsplit > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (warp >= 2) {
            const int f = (warp - 2) * 32 + lane;
            const int64_t j = j0 + f;
            const bool ok = j < p.out;
            float b[RP > 0 ? RP : 1];
            i8_load_factor<RP>(p, j, ok, b);
            const float so = (ok && p.out_scale) ? __ldg(p.out_scale + j) : 1.0f;
            const int live = min(NT, p.m - t0);              // tokens of this tile
            const int c1 = live * (part + 1) / nsplit;
            const uint32_t base = smem_u32(smem) + f * 4;
            for (int c = live * part / nsplit; c < c1; ++c) {
                int sum = 0;
#pragma unroll
                for (int r = 0; r < kI8MaxSplit; ++r) {
                    if (r < nsplit) {
                        uint32_t remote;
                        int x;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(base + c * 512), "r"(r));
                        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(remote) : "memory");
                        sum += x;
                    }
                }
                const int acc[1] = {sum};
                if (ok) i8_store<RP, 1>(p, t0 + c, j, acc, so, b);
            }
        }
        __syncwarp();
        // every CTA's shared memory stays until all have read it
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// Many tokens: a pair of CTAs computes 256 output features x NT tokens with
// tcgen05.mma.cta_group::2.  Each CTA loads its 128 features of the weight and
// its half of the tokens; the pair's tensor cores share the token halves, so
// an SM reads and stages half the token bytes per MMA that it would alone.
// The kernel is persistent (one pair per two SMs) with two accumulators in
// tensor memory: eight epilogue warps drain one while the MMAs fill the other.
// ---------------------------------------------------------------------------
constexpr int kI8PairThreads = 320;       // producer warp, MMA warp, eight epilogue warps

// RP: the adapter's rank rounded up to 0, 16 or 64; its factors of a tile are
// staged in shared memory (T as fp32 [NT][RP + 4], the other factor as bf16
// [128][RP + 4]: rows that the epilogue's reads meet without bank conflicts).
template <int NT, int RP>
struct I8PairCfg {
    static constexpr int kStages = RP > 16 ? 4 : 6;
    static constexpr int kABytes = 128 * 128;
    static constexpr int kBBytes = NT / 2 * 128;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kRow = RP + 4;
    static constexpr size_t kScale = size_t(kStages) * kStageBytes;          // token scales, fp32 [NT]
    static constexpr size_t kT = kScale + size_t(NT) * 4;
    static constexpr size_t kP = kT + (RP > 0 ? size_t(NT) * kRow * 4 : 0);
    static constexpr size_t kBar = kP + (RP > 0 ? size_t(128) * kRow * 2 : 0);
    static constexpr size_t kBytes = kBar + (2 * kStages + 4) * 8 + 16 + 1024;
    static_assert(kBytes <= 232448, "shared memory of a CTA");
};

// 16 lanes x 32 columns of 32 bits, 16 registers: lane (g, c) gets rows g
// (registers 4 i, 4 i + 1) and g + 8 (4 i + 2, 4 i + 3) at columns 8 i + 2 c
// and 8 i + 2 c + 1.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// The staged factors of a tile: s T (zero beyond the tokens and the rank) and
// the other factor of this CTA's 128 output features, by 256 threads.
template <int NT, int RP>
__device__ __forceinline__ void i8_stage_factors(const I8Params& p, int64_t j0, int t0, float* sT, uint16_t* sP, int tid) {
    constexpr int ROW = RP + 4;
    const int ru = (p.rank + 3) / 4 * 4;
    if ((p.rank & 3) == 0) {
        const int q = ru / 4;
        for (int e = tid; e < NT * q; e += 256) {
            const int t = e / q, u = (e - t * q) * 4;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (t0 + t < p.m) v = __ldg(reinterpret_cast<const float4*>(p.T + static_cast<int64_t>(t0 + t) * p.rank + u));
            v.x *= p.s, v.y *= p.s, v.z *= p.s, v.w *= p.s;
            *reinterpret_cast<float4*>(sT + t * ROW + u) = v;
        }
    } else {
        for (int e = tid; e < NT * ru; e += 256) {
            const int t = e / ru, u = e - t * ru;
            sT[t * ROW + u] =
                (t0 + t < p.m && u < p.rank) ? p.s * __ldg(p.T + static_cast<int64_t>(t0 + t) * p.rank + u) : 0.0f;
        }
    }
    if (p.pj == 1) {                         // the features are contiguous: neighbours to neighbouring threads
        for (int e = tid; e < 128 * ru; e += 256) {
            const int u = e >> 7, f = e & 127;
            sP[f * ROW + u] = (j0 + f < p.out && u < p.rank) ? __ldg(p.P + j0 + f + u * p.pu) : uint16_t(0);
        }
    } else {                                 // the ranks are
        for (int e = tid; e < 128 * ru; e += 256) {
            const int f = e / ru, u = e - f * ru;
            sP[f * ROW + u] = (j0 + f < p.out && u < p.rank) ? __ldg(p.P + (j0 + f) * p.pj + u) : uint16_t(0);
        }
    }
}

__device__ __forceinline__ uint32_t map_to_rank(uint32_t smem_addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// A tiled load into this CTA's shared memory that reports to a barrier of the
// pair's first CTA (a cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void mma_i8_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on the barrier at this offset in both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
}

template <int NT, bool TRANS, int RP>
__global__ void __launch_bounds__(kI8PairThreads, 1)
    i8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ I8Params p) {
    using C = I8PairCfg<NT, RP>;
    constexpr int S = C::kStages;
    constexpr uint32_t kTmemCols = 2 * NT;
    constexpr uint32_t kIdesc = idesc_i8_s32(256, NT, TRANS);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBar);   // used in the first CTA of the pair
    uint64_t* empty = full + S;                                     // both
    uint64_t* dfull = empty + S;                                    // both, one per accumulator
    uint64_t* dempty = dfull + 2;                                   // first CTA
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(dempty + 2);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1u;
    const int jtiles = (p.out + 255) / 256;
    const int tiles = jtiles * ((p.m + NT - 1) / NT);
    const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);
    const int nb = (p.red + 127) / 128;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 16);       // eight epilogue warps of each CTA
        }
        *s_abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(s_tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == 0) {
        // ------------------------------------------------------------ producer (each CTA its own operands)
        if (lane == 0) {
            int it = 0;
            auto load_w = [&](int i, int tile, int b) {
                const int st = i % S;
                uint8_t* a = smem + st * C::kStageBytes;
                if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * C::kStageBytes);
                const uint32_t bar = map_to_rank(smem_u32(&full[st]), 0);
                const int j0 = (tile % jtiles) * 256 + static_cast<int>(rank) * 128;
                if (TRANS) tma_load_2d_pair(a, &tmW, bar, j0, b * 128);
                else tma_load_2d_pair(a, &tmW, bar, b * 128, j0);
            };
            // weights ahead of the kernel that writes the token codes
            const int ahead = first < tiles ? (nb < S ? nb : S) : 0;
            for (int i = 0; i < ahead; ++i) load_w(i, first, i);
            griddep_wait();
            griddep_launch_dependents();
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += step) {
                const int t0 = (tile / jtiles) * NT + static_cast<int>(rank) * (NT / 2);
                for (int b = 0; b < nb; ++b, ++it) {
                    const int st = it % S;
                    if (it >= ahead) {
                        if (it >= S && !mbar_wait(&empty[st], ((it / S) - 1) & 1, s_abort)) {
                            ok = false;
                            break;
                        }
                        load_w(it, tile, b);
                    }
                    tma_load_2d_pair(smem + st * C::kStageBytes + C::kABytes, &tmX,
                                     map_to_rank(smem_u32(&full[st]), 0), b * 128, t0);
                }
            }
            // the last slots are released: no copy is in flight and no commit is
            // still on its way to this CTA
            for (int d = max(0, it - S); ok && d < it; ++d) ok = mbar_wait(&empty[d % S], (d / S) & 1, s_abort);
            if (!ok && rank == 0)
                for (int d = max(0, it - S); d < it; ++d) mbar_wait_drain(&full[d % S], (d / S) & 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (first CTA, for the pair)
        if (lane == 0 && rank == 0) {
            int it = 0, n = 0;
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += step, ++n) {
                const int buf = n & 1;
                ok = n < 2 || mbar_wait(&dempty[buf], ((n >> 1) - 1) & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(buf * NT);
                for (int b = 0; b < nb; ++b, ++it) {
                    const int st = it % S;
                    ok = mbar_wait(&full[st], (it / S) & 1, s_abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + st * C::kStageBytes);
                    const uint64_t bdesc = smem_desc_k_sw128(a + C::kABytes);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_i8_ss_pair(d, i8_a_desc<TRANS>(a, j), bdesc + static_cast<uint64_t>(2 * j), kIdesc,
                                       (b > 0 || j > 0) ? 1u : 0u);
                    mma_commit_pair(&empty[st]);
                }
                if (ok) mma_commit_pair(&dfull[buf]);
            }
            // given up: the MMAs issued so far end before tensor memory is freed
            if (!ok && it > 0) mbar_wait_drain(&empty[(it - 1) % S], ((it - 1) / S) & 1);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        griddep_wait();
        const int quarter = warp & 3, half = (warp - 2) >> 2, tid = threadIdx.x - 64;
        float* sx = reinterpret_cast<float*>(smem + C::kScale);
        float* sT = reinterpret_cast<float*>(smem + C::kT);
        uint16_t* sP = reinterpret_cast<uint16_t*>(smem + C::kP);
        int n = 0;
        for (int tile = first; tile < tiles; tile += step, ++n) {
            const int buf = n & 1;
            const int64_t j0 = static_cast<int64_t>(tile % jtiles) * 256 + static_cast<int>(rank) * 128;
            const int t0 = (tile / jtiles) * NT, h0 = half * (NT / 2);
            // the tile's scales and factors, while its MMAs run
            named_barrier_sync(1, 256);
            if (tid < NT) sx[tid] = t0 + tid < p.m ? __ldg(p.row_scale + t0 + tid) : 0.0f;
            if (RP > 0) i8_stage_factors<NT, RP>(p, j0, t0, sT, sP, tid);
            named_barrier_sync(1, 256);
            const uint32_t taddr = tmem + static_cast<uint32_t>(buf * NT + h0) + (static_cast<uint32_t>(quarter * 32) << 16);
            const int live = min(NT / 2, p.m - t0 - h0);          // tokens of this warp's half that exist
            float* y = p.Y + static_cast<int64_t>(t0 + h0) * p.out + j0 + quarter * 32;
            if (RP == 0) {
                // lane = output feature: 128 contiguous bytes per token
                const int64_t j = j0 + quarter * 32 + lane;
                const bool ok = j < p.out;
                const float so = (ok && p.out_scale) ? __ldg(p.out_scale + j) : 1.0f;
                if (!mbar_wait(&dfull[buf], (n >> 1) & 1, s_abort)) continue;   // given up: still meet at the barriers
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < NT / 2; c += 16) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(taddr + c, r);
                    tmem_ld_wait();
                    if (c + 16 >= NT / 2) {
                        // the last columns are in registers: the accumulator is free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&dempty[buf]), 0));
                    }
                    float* row = y + static_cast<int64_t>(c) * p.out + lane;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (ok && c + i < live) *row = static_cast<float>(static_cast<int>(r[i])) * sx[h0 + c + i] * so;
                        row += p.out;
                    }
                    __syncwarp();
                }
            } else {
                // lane (g, c): four features 8 apart, two tokens of every eight, so that a
                // value read from shared memory serves several outputs
                const int g = lane >> 2, c2 = (lane & 3) * 2;
                const int ru = (p.rank + 3) / 4 * 4;
                float so[4];
                bool ok[4];
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int64_t j = j0 + quarter * 32 + 8 * f + g;
                    ok[f] = j < p.out;
                    so[f] = (ok[f] && p.out_scale) ? __ldg(p.out_scale + j) : 1.0f;
                }
                if (!mbar_wait(&dfull[buf], (n >> 1) & 1, s_abort)) continue;   // given up: still meet at the barriers
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < NT / 2; c += 32) {
                    uint32_t r[2][16];
                    tmem_ld_16x256b_x4(taddr + c, r[0]);
                    tmem_ld_16x256b_x4(taddr + c + (16u << 16), r[1]);
                    float d[4][4][2];                               // [feature][token group][token]
#pragma unroll
                    for (int f = 0; f < 4; ++f)
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[f][i][0] = d[f][i][1] = 0.0f;
                    const float* tr = sT + (h0 + c + c2) * C::kRow;
                    const uint16_t* pr = sP + (quarter * 32 + g) * C::kRow;
#pragma unroll 1
                    for (int u = 0; u < ru; u += 4) {
                        float b[4][4];
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const uint2 w = *reinterpret_cast<const uint2*>(pr + 8 * f * C::kRow + u);
                            b[f][0] = __uint_as_float(w.x << 16);
                            b[f][1] = __uint_as_float(w.x & 0xFFFF0000u);
                            b[f][2] = __uint_as_float(w.y << 16);
                            b[f][3] = __uint_as_float(w.y & 0xFFFF0000u);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float4 t = *reinterpret_cast<const float4*>(tr + (8 * i + k) * C::kRow + u);
#pragma unroll
                                for (int f = 0; f < 4; ++f) {
                                    d[f][i][k] = fmaf(t.x, b[f][0], d[f][i][k]);
                                    d[f][i][k] = fmaf(t.y, b[f][1], d[f][i][k]);
                                    d[f][i][k] = fmaf(t.z, b[f][2], d[f][i][k]);
                                    d[f][i][k] = fmaf(t.w, b[f][3], d[f][i][k]);
                                }
                            }
                    }
                    tmem_ld_wait();
                    if (c + 32 >= NT / 2) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&dempty[buf]), 0));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 sxv = *reinterpret_cast<const float2*>(sx + h0 + c + 8 * i + c2);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int t = c + 8 * i + c2 + k;
                            float* row = y + static_cast<int64_t>(t) * p.out + g;
#pragma unroll
                            for (int f = 0; f < 4; ++f) {
                                const int acc = static_cast<int>(r[f >> 1][4 * i + 2 * (f & 1) + k]);
                                const float v = static_cast<float>(acc) * (k ? sxv.y : sxv.x) * so[f];
                                if (ok[f] && t < live) row[8 * f] = v + d[f][i][k];
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    // no CTA leaves while its partner may still signal it or read its memory
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

}  // namespace lbq
