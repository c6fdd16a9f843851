// i8adapter.cuh -- the adapter's product of an 8-bit layer's call, fp32 [m, r]:
//
//   forward   T = X A^T   (A [r, len], rows contiguous along the reduction)
//   backward  U = dY B    (B [len, r], the rank contiguous)
//
// Skinny (r <= 64) and bandwidth-bound.  A CTA takes MT tokens and a part of
// the reduction, in chunks of 128 through a ring of cp.async stages; its eight
// warps take 16 of each chunk's 128 steps, so a fragment of the adapter's
// factor serves all the CTA's tokens.  The products run on mma.sync (bf16 in,
// fp32 sums); the parts of a token tile form a cluster and are joined over
// distributed shared memory in a fixed order.  A warp's sum takes one product of
// 16 terms per chunk and is kept in fp32 registers outside the tensor core, whose
// own additions truncate: U over 28672 at rank 33 for 2048 tokens was off by
// 8.6e-7 rms with chains of them and is by 1.5e-7 (an fp32 product: 3.0e-7), for
// 84 us instead of 75 at 4096 x 14336, rank 36.
#pragma once

#include "common.cuh"
#include "dqgemm_bwd.cuh"
#include "lora.cuh"

namespace lbq {

constexpr int kAdThreads = 256;
constexpr int kAdChunk = 128;
constexpr int kAdMaxParts = 16;          // few tokens: clusters beyond the portable size of 8

template <int MT, int R8>
struct AdapterSmem {
    static constexpr int kStages = MT <= 16 ? 8 : 4;
    static constexpr int kRow = kAdChunk * 2 + 16;            // 272 bytes: conflict-free ldmatrix
    static constexpr int kXBytes = MT * kRow;
    static constexpr int kWBytes = 8 * R8 * kRow;             // also holds 128 rows of 2 r bytes
    static constexpr int kStageBytes = kXBytes + kWBytes;
    static constexpr int kRed = 8 * MT * 8 * R8 * 4;          // the warps' sums reuse the ring
    static constexpr int kPart = MT * 8 * R8 * 4;             // the CTA's sums, read by the cluster
    static constexpr int kRing = kStages * kStageBytes > kRed ? kStages * kStageBytes : kRed;
    static constexpr int kBytes = kRing + kPart;
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// 16 bytes to shared memory, the last 16 - n of them zero (n may be 0).
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <bool COL, int MT, int R8>
__global__ void __launch_bounds__(kAdThreads) i8_adapter_kernel(const uint16_t* __restrict__ in, int64_t m, int len,
                                                                const uint16_t* __restrict__ wt, int r,
                                                                float* __restrict__ out) {
    using L = AdapterSmem<MT, R8>;
    constexpr int NR = 8 * R8, S = L::kStages, TILES = MT / 16;
    extern __shared__ __align__(128) uint8_t ad_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int parts = static_cast<int>(gridDim.y), part = static_cast<int>(blockIdx.y);
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * MT;
    const int chunks = (len + kAdChunk - 1) / kAdChunk;
    const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * part / parts);
    const int nc = static_cast<int>(static_cast<int64_t>(chunks) * (part + 1) / parts) - c0;
    const uint32_t base = smem_u32(ad_smem);
    griddep_wait();                 // everything before this kernel is complete ...
    griddep_launch_dependents();    // ... so what follows may start beside it

    auto load_chunk = [&](int i) {
        const uint32_t sx = base + (i % S) * L::kStageBytes, sw = sx + L::kXBytes;
        const int k0 = (c0 + i) * kAdChunk;
        for (int e = threadIdx.x; e < MT * 16; e += kAdThreads) {
            const int row = e >> 4, k = k0 + (e & 15) * 8;     // len % 8 == 0: a piece is inside or outside
            const bool ok = row0 + row < m && k < len;
            cp_async16_part(sx + row * L::kRow + (e & 15) * 16, ok ? in + (row0 + row) * len + k : in, ok ? 16 : 0);
        }
        if (!COL) {
            for (int e = threadIdx.x; e < NR * 16; e += kAdThreads) {
                const int t = e >> 4, k = k0 + (e & 15) * 8;
                const bool ok = t < r && k < len;
                cp_async16_part(sw + t * L::kRow + (e & 15) * 16, ok ? wt + static_cast<int64_t>(t) * len + k : wt,
                                ok ? 16 : 0);
            }
        } else {
            // 128 rows of r ranks are one run of 256 r bytes
            const int have = min(kAdChunk, len - k0) * r * 2;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(wt + static_cast<int64_t>(k0) * r);
            for (int e = threadIdx.x; e < kAdChunk * r / 8; e += kAdThreads) {
                const int n = min(16, max(0, have - e * 16));
                cp_async16_part(sw + e * 16, n > 0 ? src + e * 16 : reinterpret_cast<const uint8_t*>(wt), n);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // a product of 16 terms by the tensor core, its addition to the sum in fp32: a tensor core's own would truncate
    float acc[TILES][R8][4];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int t = 0; t < R8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][t][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        if (i < nc) load_chunk(i);
        else asm volatile("cp.async.commit_group;" ::: "memory");
    }
    const int q = lane >> 3, l8 = lane & 7, kk = warp * 16;
    for (int i = 0; i < nc; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncthreads();                                       // chunk i landed; chunk i - 1 consumed
        if (i + S - 1 < nc) load_chunk(i + S - 1);
        else asm volatile("cp.async.commit_group;" ::: "memory");
        const uint32_t sx = base + (i % S) * L::kStageBytes, sw = sx + L::kXBytes;
        uint32_t b[R8][2];
        if (!COL) {
#pragma unroll
            for (int t = 0; t < R8; t += 2) {
                uint32_t f[4];
                const int row = t * 8 + (R8 > 1 ? (q >> 1) * 8 : 0) + l8;
                ldmatrix_x4(f, sw + row * L::kRow + (kk + (q & 1) * 8) * 2);
                b[t][0] = f[0], b[t][1] = f[1];
                if (R8 > 1) b[t + (R8 > 1)][0] = f[2], b[t + (R8 > 1)][1] = f[3];
            }
        } else if ((r & 7) == 0) {
#pragma unroll
            for (int t = 0; t < R8; t += 2) {
                uint32_t f[4];
                const int u = t * 8 + (R8 > 1 ? (q >> 1) * 8 : 0);
                // ranks past r are not stored: such a block reads the first one and is dropped
                ldmatrix_x4_trans(f, sw + ((kk + (q & 1) * 8 + l8) * r + (u < r ? u : 0)) * 2);
                const bool in0 = t * 8 < r, in1 = t * 8 + 8 < r;
                b[t][0] = in0 ? f[0] : 0u, b[t][1] = in0 ? f[1] : 0u;
                if (R8 > 1) b[t + (R8 > 1)][0] = in1 ? f[2] : 0u, b[t + (R8 > 1)][1] = in1 ? f[3] : 0u;
            }
        } else {
            const uint16_t* w = reinterpret_cast<const uint16_t*>(ad_smem + (i % S) * L::kStageBytes + L::kXBytes);
#pragma unroll
            for (int t = 0; t < R8; ++t) {
                const int u = t * 8 + g;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = kk + 8 * h + 2 * c;
                    b[t][h] = u < r ? static_cast<uint32_t>(w[k * r + u]) | (static_cast<uint32_t>(w[(k + 1) * r + u]) << 16)
                                    : 0u;
                }
            }
        }
#pragma unroll
        for (int mt = 0; mt < TILES; ++mt) {
            uint32_t a[4];
            ldmatrix_x4(a, sx + (mt * 16 + (q & 1) * 8 + l8) * L::kRow + (kk + (q >> 1) * 8) * 2);
#pragma unroll
            for (int t = 0; t < R8; ++t) {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                lora_mma(d, a[0], a[1], a[2], a[3], b[t][0], b[t][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][t][e] += d[e];
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float* red = reinterpret_cast<float*>(ad_smem);            // [8 warps][MT][NR]
    float* sum = reinterpret_cast<float*>(ad_smem + L::kRing); // [MT][NR]
#pragma unroll
    for (int mt = 0; mt < TILES; ++mt)
#pragma unroll
        for (int t = 0; t < R8; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2*>(red + (warp * MT + mt * 16 + g + 8 * h) * NR + t * 8 + 2 * c) =
                    make_float2(acc[mt][t][2 * h], acc[mt][t][2 * h + 1]);
    __syncthreads();
    for (int e = threadIdx.x; e < MT * NR; e += kAdThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += red[w * MT * NR + e];
        sum[e] = v;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int e = threadIdx.x * parts + part; e < MT * NR; e += kAdThreads * parts) {
        const int row = e / NR, t = e - row * NR;
        if (t >= r || row0 + row >= m) continue;
        float v = 0.0f;
#pragma unroll
        for (int p = 0; p < (MT <= 16 ? kAdMaxParts : 8); ++p) {
            if (p < parts) {
                uint32_t remote;
                float x;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(sum + e)), "r"(p));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(remote) : "memory");
                v += x;
            }
        }
        out[(row0 + row) * r + t] = v;
    }
    // the cluster's shared memory stays until all have read it
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Many tokens: the same product on tcgen05.  A CTA takes 128 tokens and a part
// of the reduction in blocks of 64, both operands by TMA: the tokens as the
// K-major A operand, the adapter's factor as the B operand, K-major in the
// forward and MN-major (the rank contiguous) in the backward, where its rows of
// 2 r bytes need a multiple of 16 (r % 8 == 0; other ranks take the kernel
// above).  A tensor core's addition to its accumulator truncates, so chains of
// them stay short: the blocks go to the accumulators of a bank in turn, four
// blocks (16 MMAs) each, while the epilogue warps add the other bank's to fp32
// registers, whose additions round.  (U of 2048 tokens x 28672 at rank 64: off by
// 1.2e-6 rms with chains of 75 MMAs and by 2.5e-7 so, an fp32 product by 3.0e-7;
// 38 us instead of 36.)
// HBM-bound: 4096 tokens x 14336 at rank 16 in 28 us (4.2 TB/s, 0.64 of the copy
// rate), x 4096 in 15 us from cold caches (2.3 TB/s: the start, four rounds of
// the ring and the join are of one size).
// ---------------------------------------------------------------------------
constexpr int kAdTcThreads = 192;          // producer warp, MMA warp, four epilogue warps

// The ring takes over half of the SM's shared memory: one CTA per SM.  With two
// or three, the CTAs that start early, while the product of the call before is
// still busy on the other SMs, crowd the first free ones, and the kernel lasted
// 49 instead of 28 us behind a 4096-token product (117 MB of tokens).
template <int NR>
struct AdapterTcSmem {
    static constexpr int kStages = NR <= 16 ? 7 : NR <= 32 ? 6 : 5;
    static constexpr int kXBytes = 128 * 128;
    static constexpr int kWBytes = NR * 128;
    static constexpr int kStageBytes = kXBytes + kWBytes;
    static constexpr int kSets = 128 / NR;                     // accumulators of NR columns in each of two banks
    static constexpr int kRound = 4 * kSets;                   // blocks to a bank before it is drained
    static constexpr int kRow = NR + 1;                        // the sums of a token, read by the cluster
    static constexpr size_t kBar = size_t(kStages) * kStageBytes;
    static constexpr size_t kBytes = kBar + (2 * kStages + 5) * 8 + 16 + 1024;
    static_assert(size_t(128) * kRow * 4 <= kBar, "the sums reuse the ring");
};

// MN-major B operand whose rows of NR bf16 fill one swizzle atom (32, 64 or 128
// bytes): groups of 8 reduction steps are 16 NR bytes apart.
template <int NR>
__device__ __forceinline__ uint64_t smem_desc_mn_rank(uint32_t addr) {
    constexpr uint64_t kLayout = NR == 64 ? 2 : NR == 32 ? 4 : 6;
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1u) << 16) |
           (static_cast<uint64_t>((16u * NR) >> 4) << 32) | (static_cast<uint64_t>(1u) << 46) | (kLayout << 61);
}

template <bool COL, int NR>
__global__ void __launch_bounds__(kAdTcThreads) i8_adapter_tc_kernel(const __grid_constant__ CUtensorMap tmX,
                                                                     const __grid_constant__ CUtensorMap tmW, int m,
                                                                     int len, int r, float* __restrict__ out) {
    using L = AdapterTcSmem<NR>;
    constexpr int S = L::kStages;
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, NR) | (COL ? 1u << 16 : 0u);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* empty = full + S;
    uint64_t* dfull = empty + S;        // a bank's sums are complete
    uint64_t* dempty = dfull + 2;       // a bank is drained
    uint64_t* done = dempty + 2;        // every MMA is
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = static_cast<int>(gridDim.y), part = static_cast<int>(blockIdx.y);
    const int t0 = static_cast<int>(blockIdx.x) * 128;
    const int blocks = (len + 63) / 64;
    const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * part / parts);
    const int nb = static_cast<int>(static_cast<int64_t>(blocks) * (part + 1) / parts) - b0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 4);   // four epilogue warps
        }
        mbar_init(done, 1);
        *s_abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        tmem_alloc(s_tmem, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    griddep_wait();                 // everything before this kernel is complete ...
    griddep_launch_dependents();    // ... so what follows may start beside it
    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            for (; i < nb; ++i) {
                const int st = i % S;
                if (i >= S && !mbar_wait(&empty[st], ((i / S) - 1) & 1, s_abort)) break;
                uint8_t* x = smem + st * L::kStageBytes;
                mbar_arrive_expect_tx(&full[st], L::kStageBytes);
                tma_load_2d(x, &tmX, &full[st], (b0 + i) * 64, t0);
                if (COL) tma_load_2d(x + L::kXBytes, &tmW, &full[st], 0, (b0 + i) * 64);
                else tma_load_2d(x + L::kXBytes, &tmW, &full[st], (b0 + i) * 64, 0);
            }
            for (int d = max(0, i - S); d < i; ++d) mbar_wait_drain(&full[d % S], (d / S) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // (a loop of rounds: a commit under a condition in the loop of blocks cost 2 us of 36)
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i0 = 0, rd = 0; ok && i0 < nb; i0 += L::kRound, ++rd) {
                if (rd >= 2 && !mbar_wait(&dempty[rd & 1], ((rd >> 1) - 1) & 1, s_abort)) break;
                const uint32_t bank = tmem + static_cast<uint32_t>((rd & 1) * 128);
                const int n = min(nb - i0, L::kRound);
                for (int c = 0; c < n; ++c) {
                    ok = mbar_wait(&full[st], ph, s_abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t x = smem_u32(smem + st * L::kStageBytes), w = x + L::kXBytes;
                    const uint32_t d = bank + static_cast<uint32_t>((c % L::kSets) * NR);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_ss(d, smem_desc_k_sw128(x) + static_cast<uint64_t>(2 * j),
                               COL ? smem_desc_mn_rank<NR>(w + j * 32 * NR)
                                   : smem_desc_k_sw128(w) + static_cast<uint64_t>(2 * j),
                               kIdesc, (c >= L::kSets || j > 0) ? 1u : 0u);
                    mma_commit(&empty[st]);
                    if (++st == S) st = 0, ph ^= 1u;
                }
                if (ok) mma_commit(&dfull[rd & 1]);
            }
            mma_commit(done);
            mbar_wait_drain(done, 0);
        }
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        float v[NR];
#pragma unroll
        for (int e = 0; e < NR; ++e) v[e] = 0.0f;
        const int rounds = (nb + L::kRound - 1) / L::kRound;
        bool ok = true;
#pragma unroll 1
        for (int rd = 0; rd < rounds; ++rd) {
            const int bank = rd & 1, sets = min(nb - rd * L::kRound, L::kSets);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&dfull[bank], (rd >> 1) & 1, s_abort));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < sets; ++k) {
#pragma unroll
                for (int c = 0; c < NR; c += 16) {
                    uint32_t a[16];
                    tmem_ld_32x32b_x16(taddr + bank * 128 + k * NR + c, a);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[c + e] += __uint_as_float(a[e]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dempty[bank]);
        }
        // the last bank is complete, so is every block before it: the ring is free
        if (ok) {
            float* sum = reinterpret_cast<float*>(smem) + row * L::kRow;
#pragma unroll
            for (int e = 0; e < NR; ++e) sum[e] = v[e];
        }
    }
    tc_fence_before();
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
    const int live = min(128, m - t0);
    for (int e = threadIdx.x * parts + part; e < live * r; e += kAdTcThreads * parts) {
        const int row = e / r, t = e - row * r;
        const uint32_t at = smem_u32(smem) + (row * L::kRow + t) * 4;
        float v = 0.0f;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (p < parts) {
                uint32_t remote;
                float x;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(p));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(remote) : "memory");
                v += x;
            }
        }
        out[static_cast<int64_t>(t0) * r + e] = v;
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace lbq
