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

#include <type_traits>

#include "common.cuh"
#include "dqgemm.cuh"
#include "dqgemm_bwd.cuh"
#include "i8quant.cuh"

namespace lbq {

constexpr int kI8MaxReduction = 131072;   // 127^2 * 131072 < 2^31

struct I8Params {
    int m, out, red;           // tokens, output features, reduction length
    // row_scale and T are written by kernels of the same call while this one may be resident already: they are read
    // after griddep_wait and not through the read-only path (__ldcg); the others are complete before it starts
    const float* row_scale;    // [m] token scales
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

// ---------------------------------------------------------------------------
// Few tokens: one CTA per 128 output features x nt tokens x part of the
// reduction.  The CTAs of a cluster hold the parts of one tile; each adds up
// its share of the tokens over the cluster's shared memory.  nt is any multiple
// of 16 up to 256, so that a ragged batch multiplies few empty tokens.
// HBM-bound by the weight; the ring's blocks (16 KB of weight and nt x 128
// bytes of tokens) in flight cover the latency.  Measured: a whole call of
// 1 token x 4096 x 4096 in 8.2 us (the weight alone is 2.6 us at the copy rate),
// of 16 tokens x 4096 x 14336 at rank 16 in 18.5 us, where this kernel streams
// the 59 MB of codes at about 4.3 TB/s and the rest is the chain of three
// launches, both with L2 flushed before the call; of 512 x 4096 x 4096 at rank 16 in 29 us.
// ---------------------------------------------------------------------------
constexpr int kI8SplitThreads = 192;      // producer warp, MMA warp, four epilogue warps
constexpr int kI8MaxSplit = 8;
constexpr int kI8SplitMaxStages = 12;

// Shared memory of a CTA: the ring (the partial sums reuse it), the token
// scales, s T of the CTA's share of the tokens, the barriers.  Tiles of more
// than 128 tokens take over half of the SM's, whatever their ring: CTAs of 256
// tensor memory columns that wait for one another in clusters must not meet
// three to an SM, where one could wait for columns that only its partner's
// partner frees.  (With at most 128 columns each, shared memory admits no more
// CTAs than the 512 columns hold, beside this library's other kernels too.)
struct I8SplitShape {
    int nt, stages, tok;
    __host__ __device__ int stage_bytes() const { return 128 * 128 + nt * 128; }
    __host__ __device__ int ring() const {
        const int sums = (nt * 512 + 1023) / 1024 * 1024;
        return stages * stage_bytes() > sums ? stages * stage_bytes() : sums;
    }
    __host__ __device__ size_t bytes(int rp) const {
        const size_t b = static_cast<size_t>(ring()) + nt * 4 + static_cast<size_t>(tok) * rp * 4 + (2 * stages + 1) * 8 + 16 + 1024;
        return nt > 128 && b < 116 * 1024 ? 116 * 1024 : b;
    }
};

template <bool TRANS, int RP>
__global__ void __launch_bounds__(kI8SplitThreads)
    i8_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ I8Params p, const I8SplitShape sh) {
    const int NT = sh.nt, S = sh.stages, stage_bytes = sh.stage_bytes();
    const uint32_t kTmemCols = tmem_cols_for(NT);
    const uint32_t kIdesc = idesc_i8_s32(128, NT, TRANS);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* sx = reinterpret_cast<float*>(smem + sh.ring());
    float* sT = sx + NT;                                     // [tok][RP]
    uint64_t* full = reinterpret_cast<uint64_t*>(sT + sh.tok * RP);
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
            auto load_w = [&](int i, int st) {
                uint8_t* a = smem + st * stage_bytes;
                mbar_arrive_expect_tx(&full[st], stage_bytes);
                if (TRANS) tma_load_2d(a, &tmW, &full[st], j0, (b0 + i) * 128);
                else tma_load_2d(a, &tmW, &full[st], (b0 + i) * 128, j0);
            };
            // the weight does not depend on the kernel before this one (which
            // starts only after everything before it is complete), the codes
            // of the tokens do
            const int ahead = nb < S ? nb : S;
            for (int i = 0; i < ahead; ++i) load_w(i, i);
            griddep_wait();
            griddep_launch_dependents();
            int i = 0, st = 0;
            uint32_t ph = 1;                                 // the first pass over the ring does not wait
            for (; i < nb; ++i) {
                if (i >= S) {
                    if (!mbar_wait(&empty[st], ph, s_abort)) break;
                    load_w(i, st);
                }
                tma_load_2d(smem + st * stage_bytes + 128 * 128, &tmX, &full[st], (b0 + i) * 128, t0);
                if (++st == S) st = 0, ph ^= 1u;
            }
            for (int d = max(0, i - S); d < i; ++d) mbar_wait_drain(&full[d % S], (d / S) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int st = 0;
            uint32_t ph = 0;
            for (int i = 0; i < nb; ++i) {
                if (!mbar_wait(&full[st], ph, s_abort)) break;
                tc_fence_after();
                const uint32_t a = smem_u32(smem + st * stage_bytes);
                const uint64_t bdesc = smem_desc_k_sw128(a + 128 * 128);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_i8_ss(tmem, i8_a_desc<TRANS>(a, j), bdesc + static_cast<uint64_t>(2 * j), kIdesc,
                              (i > 0 || j > 0) ? 1u : 0u);
                mma_commit(&empty[st]);
                if (++st == S) st = 0, ph ^= 1u;
            }
            mma_commit(dfull);
            mbar_wait_drain(dfull, 0);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int tid = threadIdx.x - 64, quarter = warp & 3;
        const int live = min(NT, p.m - t0);                  // tokens of this tile
        const int lo = live * part / nsplit, hi = live * (part + 1) / nsplit;   // this CTA's share of them
        // this thread's output feature, its scale and adapter factors
        const int f = quarter * 32 + lane;
        const int64_t j = j0 + f;
        const bool ok = j < p.out;
        griddep_wait();
        for (int t = tid; t < live; t += 128) sx[t] = __ldcg(p.row_scale + t0 + t);
        if (RP > 0) {
            const float* trow = p.T + static_cast<int64_t>(t0 + lo) * p.rank;
            constexpr int Q = RP > 0 ? RP / 4 : 1;                // 16-byte pieces of a row of sT
            if ((p.rank & 3) == 0) {
#pragma unroll 4
                for (int e = tid; e < (hi - lo) * Q; e += 128) {
                    const int t = e / Q, u = (e % Q) * 4;
                    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (u < p.rank) x = __ldcg(reinterpret_cast<const float4*>(trow + static_cast<int64_t>(t) * p.rank + u));
                    reinterpret_cast<float4*>(sT)[e] = make_float4(p.s * x.x, p.s * x.y, p.s * x.z, p.s * x.w);
                }
            } else {
#pragma unroll 8
                for (int e = tid; e < (hi - lo) * RP; e += 128) {
                    const int t = e / (RP > 0 ? RP : 1), u = e % (RP > 0 ? RP : 1);
                    sT[e] = u < p.rank ? p.s * __ldcg(trow + static_cast<int64_t>(t) * p.rank + u) : 0.0f;
                }
            }
        }
        const float so = (ok && p.out_scale) ? __ldg(p.out_scale + j) : 1.0f;
        f32x2 b[RP > 0 ? RP / 2 : 1];
        if (RP > 0) {
            auto factor = [&](int u) {
                return (ok && u < p.rank) ? bf16_bits_to_f32(__ldg(p.P + j * p.pj + u * p.pu)) : 0.0f;
            };
#pragma unroll
            for (int u = 0; u < RP; u += 2) b[u / 2] = pack2(factor(u), factor(u + 1));
        }
        named_barrier_sync(1, 128);
        // consecutive tokens from t (of this CTA's share) with their sums
        auto store = [&](int t, auto& acc, int n) {
            float* y = p.Y + static_cast<int64_t>(t0 + t) * p.out + j;
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(acc) / sizeof(int)); ++i) {
                if (i < n) {
                    float v = static_cast<float>(acc[i]) * sx[t + i] * so;
                    if (RP > 0) {
                        // All RP ranks (zeros beyond the rank) in four sums: with few warps per
                        // scheduler a branch per 16 bytes waits for every load, and one sum for
                        // every addition (904 tokens x 3508 x 224, rank 64: 61 us so, 72 with the
                        // branches, 88 with one sum too)
                        f32x2 d0 = 0, d1 = 0;
                        const float4* tr = reinterpret_cast<const float4*>(sT + (t - lo + i) * RP);
#pragma unroll
                        for (int u = 0; u < RP; u += 4) {
                            const float4 x = tr[u / 4];
                            d0 = fma2(pack2(x.x, x.y), b[u / 2], d0);
                            d1 = fma2(pack2(x.z, x.w), b[u / 2 + 1], d1);
                        }
                        const float2 e0 = unpack2(d0), e1 = unpack2(d1);
                        v += (e0.x + e0.y) + (e1.x + e1.y);
                    }
                    if (ok) *y = v;
                    y += p.out;
                }
            }
        };
        const bool done = mbar_wait(dfull, 0, s_abort);
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        if (nsplit == 1) {
#pragma unroll 1
            for (int c = 0; done && c < live; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c, r);
                tmem_ld_wait();
                int acc[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = static_cast<int>(r[i]);
                store(c, acc, live - c);
                __syncwarp();
            }
        } else {
            // this part's sums to shared memory: [token][feature]
            int* buf = reinterpret_cast<int*>(smem);
#pragma unroll 1
            for (int c = 0; done && c < live; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) buf[(c + i) * 128 + f] = static_cast<int>(r[i]);
            }
            tc_fence_before();
            __syncwarp();
            asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
            // the cluster's sums of U tokens at a time, the next ones on their way meanwhile:
            // about 32 loads in flight whatever the number of parts
            const uint32_t base = smem_u32(smem) + f * 4;
            auto join = [&](auto u_, auto parts_) {
                constexpr int U = decltype(u_)::value, PARTS = decltype(parts_)::value;
                int x[PARTS][U];
                auto fetch = [&](int c) {
#pragma unroll
                    for (int r = 0; r < PARTS; ++r) {
                        if (r < nsplit) {
                            uint32_t remote;
                            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(base + c * 512), "r"(r));
#pragma unroll
                            for (int i = 0; i < U; ++i)
                                if (c + i < hi)
                                    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x[r][i]) : "r"(remote + i * 512) : "memory");
                        }
                    }
                };
                if (lo < hi) fetch(lo);
#pragma unroll 1
                for (int c = lo; c < hi; c += U) {
                    int acc[U];
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        acc[i] = 0;
#pragma unroll
                        for (int r = 0; r < PARTS; ++r)
                            if (r < nsplit && c + i < hi) acc[i] += x[r][i];
                    }
                    if (c + U < hi) fetch(c + U);
                    store(c, acc, hi - c);
                }
            };
            using std::integral_constant;
            if (nsplit <= 2) join(integral_constant<int, 16>{}, integral_constant<int, 2>{});
            else if (nsplit <= 4) join(integral_constant<int, 8>{}, integral_constant<int, 4>{});
            else join(integral_constant<int, 4>{}, integral_constant<int, 8>{});
        }
    }
    tc_fence_before();
    __syncwarp();
    if (nsplit > 1) {
        // the producer and MMA warps meet the epilogue's first cluster barrier here
        if (warp < 2)
            asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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
// Many tokens: a pair of CTAs computes 256 output features x 256 tokens with
// tcgen05.mma.cta_group::2.  Each CTA loads its 128 features of the weight and
// its half of the tokens; the pair's tensor cores share the token halves, so
// an SM reads and stages half the token bytes per MMA that it would alone.
// Loads alone and MMAs alone each take nearly as long as both together, so
// shared memory and L2 are left to them: the adapter's term is not formed from
// shared memory by the epilogue (that took 49 us of a 219 us forward of 4096
// tokens x 14336 x 4096 at rank 16) but by the tensor cores too, in fp32.  s T is
// split there into three bf16 parts that add up to it exactly (8 + 8 + 8 bits),
// so the term is as exact as in fp32.
//
// The kernel is persistent (one pair per two SMs), with two accumulators in
// tensor memory: eight epilogue warps drain one while the MMAs fill the other.
// With an adapter the epilogue first takes the int32 sums to registers; the
// term's MMAs then write fp32 over them, issued between two blocks of the next
// tile, so that the tensor cores never wait for the epilogue.
// Dealing out the last waves' tiles in equal parts of their reduction was
// measured too: 3% less time for a reduction of 14336, 3 to 8% more for 4096.
//
// Measured at 4096 tokens, rank 16: forward to 14336 features from 4096 198 us
// (2.43 P operations/s; 235 MB of output: its stores cost about 23 us), backward
// to 4096 features from 14336 179 us (2.69 P).  MMAs alone run at 2.9 to 3.1 P at the
// clock that the power limit leaves (about 1.65 GHz), loads alone at 2.8 P.  With
// an adapter an epilogue thread holds 128 sums while the term is formed and spills
// 96 bytes of its 168 registers' worth.
// ---------------------------------------------------------------------------
constexpr int kI8PairThreads = 320;       // producer warp, MMA warp, eight epilogue warps
constexpr int kI8Tile = 256;              // output features and tokens of a pair's tile

// RP: the adapter's rank rounded up to 0, 16 or 64.  Its operands are K-major
// tiles of 128-byte rows (128-byte swizzle): P [128 features][rank], and s T
// [128 tokens] with the three parts side by side (RP 16) or in tiles of their
// own (RP 64).
template <int RP>
struct I8PairCfg {
    static constexpr int kStages = RP > 16 ? 5 : 6;
    static constexpr int kOperand = 128 * 128;                               // also an adapter tile
    static constexpr int kStageBytes = 2 * kOperand;
    static constexpr size_t kP = size_t(kStages) * kStageBytes;
    static constexpr size_t kT = kP + (RP > 0 ? kOperand : 0);
    static constexpr size_t kScale = kT + (RP > 16 ? 3 : RP > 0 ? 1 : 0) * kOperand;   // token scales, fp32 [8 warps][128]
    static constexpr size_t kBar = kScale + (RP > 0 ? 0 : 4096);
    static constexpr size_t kBytes = kBar + (2 * kStages + 6) * 8 + 16 + 1024;
    static_assert(kBytes <= 232448, "shared memory of a CTA");
};

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

__device__ __forceinline__ void mma_bf16_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// mbar_wait for arrivals from the other CTA of the pair too: acquires at cluster
// scope.  (A separate fence.acq_rel.cluster after the wait cost the MMA issuer
// 1.5 us a tile.)
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
    auto test = [&](uint32_t sleep_ns) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(sleep_ns)
            : "memory");
        return ok != 0;
    };
    if (test(0u)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 0; it < kWaitLimitIters; ++it) {
        if (test(20000u)) return true;
        if (*abort) return false;
        if ((it & 63u) == 63u && globaltimer_ns() - t0 > kWaitLimitNs) break;
    }
    *abort = 1;
    record_status(kStatusTimeout);
    return false;
}

// Arrive on the barrier at this offset in both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// The two halves of a register pair's top bf16 parts, and what is left of them:
// truncated, so that three of them hold an fp32 value exactly.  An infinity or
// a NaN leaves nothing.
__device__ __forceinline__ uint32_t i8_split_part(float& a, float& b) {
    const uint32_t ua = __float_as_uint(a) & 0xFFFF0000u, ub = __float_as_uint(b) & 0xFFFF0000u;
    const uint32_t w = (ua >> 16) | ub;
    a = (ua & 0x7F800000u) == 0x7F800000u ? 0.0f : a - __uint_as_float(ua);
    b = (ub & 0x7F800000u) == 0x7F800000u ? 0.0f : b - __uint_as_float(ub);
    return w;
}

// The adapter operands of a tile for this CTA: P of 128 features from j0, s T of
// 128 tokens from t0 (zero beyond the sizes and the rank), by 256 threads.
template <int RP>
__device__ __forceinline__ void i8_stage_factors(const I8Params& p, int64_t j0, int t0, uint8_t* sP, uint8_t* sT, int tid) {
    constexpr int UNITS = RP / 8;                       // 16-byte units of a row
    for (int e = tid; e < 128 * UNITS; e += 256) {
        const int t = e / UNITS, un = e % UNITS, u0 = un * 8;
        float v[8];
        const float* row = p.T + static_cast<int64_t>(t0 + t) * p.rank + u0;
        if (t0 + t < p.m && (p.rank & 3) == 0) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (u0 + 4 * q < p.rank) x = __ldcg(reinterpret_cast<const float4*>(row + 4 * q));
                v[4 * q] = x.x, v[4 * q + 1] = x.y, v[4 * q + 2] = x.z, v[4 * q + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = (t0 + t < p.m && u0 + u < p.rank) ? __ldcg(row + u) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] *= p.s;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            uint4 w;
            w.x = i8_split_part(v[0], v[1]);
            w.y = i8_split_part(v[2], v[3]);
            w.z = i8_split_part(v[4], v[5]);
            w.w = i8_split_part(v[6], v[7]);
            const int unit = RP <= 16 ? part * 2 + un : un;
            *reinterpret_cast<uint4*>(sT + (RP <= 16 ? 0 : part * 16384) + t * 128 + ((unit ^ (t & 7)) << 4)) = w;
        }
    }
    for (int e = tid; e < 128 * UNITS; e += 256) {
        // neighbouring threads take what is contiguous: the features (backward) or the ranks
        const int f = p.pj == 1 ? e & 127 : e / UNITS, un = p.pj == 1 ? e >> 7 : e % UNITS;
        const int64_t j = j0 + f;
        const uint16_t* src = p.P + j * p.pj;
        uint4 w;
        if (p.pj != 1 && (p.rank & 7) == 0) {
            w = make_uint4(0u, 0u, 0u, 0u);
            if (j < p.out && un * 8 < p.rank) w = __ldg(reinterpret_cast<const uint4*>(src + un * 8));
        } else {
            uint32_t h[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                h[u] = (j < p.out && un * 8 + u < p.rank) ? __ldg(src + (un * 8 + u) * p.pu) : 0u;
            w = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
        }
        *reinterpret_cast<uint4*>(sP + f * 128 + ((un ^ (f & 7)) << 4)) = w;
    }
}

template <bool TRANS, int RP>
__global__ void __launch_bounds__(kI8PairThreads, 1)
    i8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ I8Params p) {
    using C = I8PairCfg<RP>;
    constexpr int S = C::kStages;
    constexpr uint32_t kIdesc = idesc_i8_s32(256, kI8Tile, TRANS), kIdescF = idesc_bf16_f32(256, kI8Tile);
    constexpr int kTermBlock = 5;           // the term of a tile follows this block of the next one
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sP = smem + C::kP;
    uint8_t* sT = smem + C::kT;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBar);   // used in the first CTA of the pair
    uint64_t* empty = full + S;                                     // both
    uint64_t* dfull = empty + S;                                    // both: sums of a buffer complete
    uint64_t* dempty = dfull + 2;                                   // first CTA: buffer drained
    uint64_t* tready = dempty + 2;                                  // first CTA: term's operands staged, sums taken
    uint64_t* tfull = tready + 1;                                   // both: term complete
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tfull + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1u;
    const int jtiles = (p.out + kI8Tile - 1) / kI8Tile;
    const int tiles = jtiles * ((p.m - 1) / kI8Tile + 1);      // any m up to 2^31 - 1: nothing is added to it
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
        mbar_init(tready, 16);
        mbar_init(tfull, 1);
        *s_abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(s_tmem)), "r"(512) : "memory");
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
                const int j0 = (tile % jtiles) * kI8Tile + static_cast<int>(rank) * 128;
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
                const int t0 = (tile / jtiles) * kI8Tile + static_cast<int>(rank) * 128;
                for (int b = 0; b < nb; ++b, ++it) {
                    const int st = it % S;
                    if (it >= ahead) {
                        if (it >= S && !mbar_wait(&empty[st], ((it / S) - 1) & 1, s_abort)) {
                            ok = false;
                            break;
                        }
                        load_w(it, tile, b);
                    }
                    tma_load_2d_pair(smem + st * C::kStageBytes + C::kOperand, &tmX, map_to_rank(smem_u32(&full[st]), 0),
                                     b * 128, t0);
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
            // the adapter's term of the pair's n-th tile
            auto term = [&](int i) {
                if (!mbar_wait_cluster(tready, i & 1, s_abort)) return false;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>((i & 1) * kI8Tile);
                const uint64_t pd = smem_desc_k_sw128(smem_u32(sP));
                for (int part = 0; part < 3; ++part) {
                    const uint64_t td = smem_desc_k_sw128(smem_u32(sT) + (RP <= 16 ? part * 32 : part * 16384));
                    for (int k = 0; k * 16 < p.rank; ++k)
                        mma_bf16_ss_pair(d, pd + static_cast<uint64_t>(2 * k), td + static_cast<uint64_t>(2 * k), kIdescF,
                                         (part > 0 || k > 0) ? 1u : 0u);
                }
                mma_commit_pair(tfull);
                return true;
            };
            for (int tile = first; ok && tile < tiles; tile += step, ++n) {
                const int buf = n & 1;
                ok = n < 2 || mbar_wait_cluster(&dempty[buf], ((n >> 1) - 1) & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(buf * kI8Tile);
                for (int b = 0; b < nb; ++b, ++it) {
                    const int st = it % S;
                    ok = mbar_wait(&full[st], (it / S) & 1, s_abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + st * C::kStageBytes);
                    const uint64_t bdesc = smem_desc_k_sw128(a + C::kOperand);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_i8_ss_pair(d, i8_a_desc<TRANS>(a, j), bdesc + static_cast<uint64_t>(2 * j), kIdesc,
                                       (b > 0 || j > 0) ? 1u : 0u);
                    mma_commit_pair(&empty[st]);
                    if (RP > 0 && n > 0 && b == min(kTermBlock, nb - 1)) {
                        ok = term(n - 1);
                        if (!ok) break;
                    }
                }
                if (ok) mma_commit_pair(&dfull[buf]);
            }
            if (RP > 0 && ok && n > 0) ok = term(n - 1);
            // given up: the MMAs issued so far end before tensor memory is freed
            if (!ok && it > 0) mbar_wait_drain(&empty[(it - 1) % S], ((it - 1) / S) & 1);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // lane = output feature: 128 contiguous bytes of Y per token; a warp takes
        // 32 features and half of the tokens.  Y is stored to leave L2 first: the
        // weight is read again for every 256 tokens
        griddep_wait();
        const int quarter = warp & 3, half = (warp - 2) >> 2, tid = threadIdx.x - 64;
        float* sx = reinterpret_cast<float*>(smem + C::kScale) + (warp - 2) * 128;   // the warp's copy (no adapter)
        auto arrive = [&](uint64_t* bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(bar), 0));
        };
        int n = 0;
        for (int tile = first; tile < tiles; tile += step, ++n) {
            const int buf = n & 1;
            // the term's operands, while the sums are still being formed (the last tile's term,
            // which read the same shared memory, is complete: the warp has waited for it)
            if (RP > 0) {
                i8_stage_factors<(RP > 0 ? RP : 16)>(
                    p, static_cast<int64_t>(tile % jtiles) * kI8Tile + static_cast<int>(rank) * 128,
                    (tile / jtiles) * kI8Tile + static_cast<int>(rank) * 128, sP, sT, tid);
                fence_proxy_async_smem();
            }
            const int64_t j = static_cast<int64_t>(tile % jtiles) * kI8Tile + static_cast<int>(rank) * 128 + quarter * 32 + lane;
            const int t0 = (tile / jtiles) * kI8Tile + half * 128;
            const int live = min(128, p.m - t0);              // tokens of this warp's half that exist
            const bool ok = j < p.out;
            const float so = (ok && p.out_scale) ? __ldg(p.out_scale + j) : 1.0f;
            float sv[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) sv[q] = q * 32 + lane < live ? __ldcg(p.row_scale + t0 + q * 32 + lane) : 0.0f;
            float* row = p.Y + static_cast<int64_t>(t0) * p.out + j;
            const uint32_t taddr = tmem + static_cast<uint32_t>(buf * kI8Tile + half * 128) + (static_cast<uint32_t>(quarter * 32) << 16);
            if (!mbar_wait(&dfull[buf], (n >> 1) & 1, s_abort)) break;
            tc_fence_after();
            if (RP == 0) {
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 4; ++q) sx[q * 32 + lane] = sv[q];
                __syncwarp();
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(taddr + c, r);
                    tmem_ld_wait();
                    if (c == 96) arrive(&dempty[buf]);        // the last columns are in registers
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (ok && c + i < live) __stcs(row, static_cast<float>(static_cast<int>(r[i])) * sx[c + i] * so);
                        row += p.out;
                    }
                    __syncwarp();
                }
            } else {
                uint32_t r[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(taddr + 32 * q, r[q]);
                tmem_ld_wait();
                arrive(tready);
                // scaled while the term's MMAs run
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        r[q][i] = __float_as_uint(static_cast<float>(static_cast<int>(r[q][i])) *
                                                  __shfl_sync(0xFFFFFFFFu, sv[q], i) * so);
                if (!mbar_wait(tfull, n & 1, s_abort)) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t d[32];
                    tmem_ld_32x32b_x32(taddr + 32 * q, d);
                    tmem_ld_wait();
                    if (q == 3) arrive(&dempty[buf]);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (ok && 32 * q + i < live) __stcs(row, __uint_as_float(r[q][i]) + __uint_as_float(d[i]));
                        row += p.out;
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
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

}  // namespace lbq
