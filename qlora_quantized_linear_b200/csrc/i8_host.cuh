// i8_host.cuh -- host side of the 8-bit integer products: argument checks, the
// choice of kernel and split, tensor maps and launches.  Included by lbq.cu
// inside its anonymous namespace.

// Raises a kernel's limits (shared memory to what its own leaves of the 227 KB,
// clusters of more than 8) once per device; doing it again, from another thread
// too, changes nothing.
template <auto Kern>
bool raise_limits(int dev) {
    static std::atomic<uint64_t> raised{0};
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev <= 63 && (raised.load(std::memory_order_relaxed) & bit)) return true;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, Kern) != cudaSuccess ||
        cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             227 * 1024 - static_cast<int>(fa.sharedSizeBytes)) != cudaSuccess ||
        cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    raised.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Launch with optional cluster size and programmatic stream serialisation
// (the kernel waits with griddepcontrol.wait before it reads what the kernel
// before it wrote).
template <auto Kern, typename... Args>
lbq_status launch_overlapped(dim3 grid, int threads, size_t smem, dim3 cluster, cudaStream_t st, const Args&... args) {
    if (smem > 48 * 1024 || cluster.x * cluster.y * cluster.z > 8) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || !raise_limits<Kern>(dev)) return LBQ_ECUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster.x * cluster.y * cluster.z > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster.x;
        attr[1].val.clusterDim.y = cluster.y;
        attr[1].val.clusterDim.z = cluster.z;
        cfg.numAttrs = 2;
    }
    if (cudaLaunchKernelEx(&cfg, Kern, args...) != cudaSuccess) {
        (void)cudaGetLastError();
        return LBQ_ECUDA;
    }
    return LBQ_OK;
}

// How many clusters of `parts` CTAs (at most 16; 0 of more than 8 where no group
// of SMs has room for one) run at the same time, per_sm (1 or 2) CTAs to an SM: a
// cluster stays within a group of SMs, and the groups are of several sizes, so
// clusters leave SMs over.  (Sixteen clusters of 8 do not fit one CTA per SM: the
// adapter product of 2048 tokens x 28672 at rank 16 took two waves, 55 us, and
// takes one of 16 clusters of 6, 36 us.)  Asked once per device, for a kernel of
// no tensor memory with that much shared memory: the answer for one that has it
// counted a single CTA per SM.
int clusters_that_fit(int parts, int per_sm, int sms) {
    static std::atomic<int> known[16][2][kAdMaxParts + 1];      // one more than the answer, 0 until it is asked
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return per_sm * sms / parts;
    std::atomic<int>* slot = dev < 16 ? &known[dev][per_sm - 1][parts] : nullptr;
    if (slot && (n = slot->load(std::memory_order_relaxed)) > 0) return n - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, static_cast<unsigned>(parts));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = (per_sm == 1 ? 116 : 106) * 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = static_cast<unsigned>(parts);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    constexpr auto kern = i8_quantize_rows_kernel<kSrcBf16, false, false, 1, 256>;
    const bool asked = raise_limits<kern>(dev) && cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess;
    if (!asked) (void)cudaGetLastError();
    // clusters of 8 are portable: any GPU runs one
    if (parts > 8) n = asked ? n : 0;
    else if (!asked || n < 1) n = std::max(1, per_sm * sms / parts);
    if (slot) slot->store(n + 1, std::memory_order_relaxed);
    return n;
}

// The largest number of parts up to `most` whose clusters, `count` of them, run
// at the same time.
int parts_that_fit(int64_t most, int64_t count, int per_sm, int sms) {
    int parts = static_cast<int>(most);
    while (parts > 1 && clusters_that_fit(parts, per_sm, sms) < count) --parts;
    return parts;
}

lbq_status check_i8weight(const lbq_i8weight* q, bool need_data) {
    if (!q) return LBQ_EINVAL;
    if (q->n < 1 || q->k < 16 || q->k % 16 != 0 || q->k > kI8MaxReduction) return LBQ_EINVAL;
    if (need_data) {
        if (!q->codes || !q->scale) return LBQ_EINVAL;
        if (!aligned16(q->codes) || !aligned16(q->scale)) return LBQ_EALIGN;
    }
    return LBQ_OK;
}

// ---------------------------------------------------------------------------
// rows to codes
// ---------------------------------------------------------------------------
template <int SRC, bool SCALED, bool BESIDE>
lbq_status run_i8_quantize(const void* in, int64_t rows, int64_t len, const float* chan, int8_t* codes, int64_t ldc,
                           float* scale, int sms, cudaStream_t st) {
#define LBQ_I8_ROWS(NV, THREADS)                                                                                       \
    launch_overlapped<i8_quantize_rows_kernel<SRC, SCALED, BESIDE, NV, THREADS>>(                                      \
        dim3(static_cast<unsigned>(rows)), THREADS, 0, dim3(1, 1, 1), st, in, len, chan, codes, ldc, scale)
    const int64_t nvec = len / 8;
    if (SRC == kSrcBf16 && rows < 2 * sms) {
        // few rows: latency, so a piece or two per thread
        if (nvec <= 256) return LBQ_I8_ROWS(1, 256);
        if (nvec <= 512) return LBQ_I8_ROWS(1, 512);
        if (nvec <= 1024) return LBQ_I8_ROWS(1, 1024);
        if (nvec <= 2048) return LBQ_I8_ROWS(2, 1024);
    } else {
        // many rows: fewer threads with more pieces each (4096 x 4096: 10 us with 128
        // threads, 16 with 512; 4096 x 14336: 28 with 256, 32 with 512, 40 with 1024)
        if (nvec <= 256) return LBQ_I8_ROWS(2, 128);
        if (nvec <= 512) return LBQ_I8_ROWS(4, 128);
        if (nvec <= 1024) return LBQ_I8_ROWS(4, 256);
        if (nvec <= 1792) return LBQ_I8_ROWS(7, 256);
        if (nvec <= 2048) return LBQ_I8_ROWS(4, 512);
        if (nvec <= 3584) return LBQ_I8_ROWS(7, 512);
    }
    if (nvec <= 4096) return LBQ_I8_ROWS(4, 1024);
    return LBQ_I8_ROWS(0, 1024);
#undef LBQ_I8_ROWS
}

template <bool COL, int MT, int R8>
lbq_status launch_i8_adapter(const void* in, int64_t m, int64_t len, const void* wt, int r, float* out, int sms,
                             cudaStream_t st) {
    // one token tile: as many parts as a cluster holds on this GPU; more: parts that fill the SMs
    const int64_t groups = cdiv(m, MT), chunks = cdiv(len, kAdChunk);
    constexpr int kPerSm = AdapterSmem<MT, R8>::kBytes <= 106 * 1024 ? 2 : 1;
    const int64_t parts =
        MT <= 16 ? parts_that_fit(std::min<int64_t>(kAdMaxParts, chunks), 1, 1, sms)
                 : parts_that_fit(std::min<int64_t>({8, chunks, std::max<int64_t>(1, kPerSm * sms / groups)}), groups, kPerSm, sms);
    return launch_overlapped<i8_adapter_kernel<COL, MT, R8>>(
        dim3(static_cast<unsigned>(groups), static_cast<unsigned>(parts)), kAdThreads, AdapterSmem<MT, R8>::kBytes,
        dim3(1, static_cast<unsigned>(parts), 1), st, static_cast<const uint16_t*>(in), m, static_cast<int>(len),
        static_cast<const uint16_t*>(wt), r, out);
}

template <bool COL, int NR>
lbq_status launch_i8_adapter_tc(const void* in, int64_t m, int64_t len, const void* wt, int r, float* out, int sms,
                                cudaStream_t st) {
    CUtensorMap tmX, tmW;
    if (!make_map_2d(&tmX, in, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, m, len, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B))
        return LBQ_ECUDA;
    const bool ok = COL ? make_map_2d(&tmW, wt, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, len, r, 64, NR,
                                      NR == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                      : NR == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                 : CU_TENSOR_MAP_SWIZZLE_32B)
                        : make_map_2d(&tmW, wt, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, len, NR, 64,
                                      CU_TENSOR_MAP_SWIZZLE_128B);
    if (!ok) return LBQ_ECUDA;
    const int64_t groups = cdiv(m, 128), blocks = cdiv(len, 64);
    const int64_t parts = parts_that_fit(std::min<int64_t>({8, blocks, std::max<int64_t>(1, sms / groups)}), groups, 1, sms);
    return launch_overlapped<i8_adapter_tc_kernel<COL, NR>>(
        dim3(static_cast<unsigned>(groups), static_cast<unsigned>(parts)), kAdTcThreads, AdapterTcSmem<NR>::kBytes,
        dim3(1, static_cast<unsigned>(parts), 1), st, tmX, tmW, static_cast<int>(m), static_cast<int>(len), r, out);
}

template <bool COL>
lbq_status run_i8_adapter_tc(const void* in, int64_t m, int64_t len, const void* wt, int r, float* out, int sms,
                             cudaStream_t st) {
    if (r <= 16) return launch_i8_adapter_tc<COL, 16>(in, m, len, wt, r, out, sms, st);
    if (r <= 32) return launch_i8_adapter_tc<COL, 32>(in, m, len, wt, r, out, sms, st);
    return launch_i8_adapter_tc<COL, 64>(in, m, len, wt, r, out, sms, st);
}

template <bool COL, int MT>
lbq_status run_i8_adapter(const void* in, int64_t m, int64_t len, const void* wt, int r, float* out, int sms,
                          cudaStream_t st) {
    if (r <= 8) return launch_i8_adapter<COL, MT, 1>(in, m, len, wt, r, out, sms, st);
    if (r <= 16) return launch_i8_adapter<COL, MT, 2>(in, m, len, wt, r, out, sms, st);
    if (r <= 32) return launch_i8_adapter<COL, MT, 4>(in, m, len, wt, r, out, sms, st);
    return launch_i8_adapter<COL, MT, 8>(in, m, len, wt, r, out, sms, st);
}

// The adapter's product of the tokens.
template <bool BWD>
lbq_status run_i8_factor(const void* in, int64_t m, int64_t len, const void* wt, int r, float* out, int sms,
                         cudaStream_t st) {
    if (m <= 16) return run_i8_adapter<BWD, 16>(in, m, len, wt, r, out, sms, st);
    if constexpr (BWD) {
        if (r % 8 != 0) return run_i8_adapter<true, 64>(in, m, len, wt, r, out, sms, st);
    }
    return run_i8_adapter_tc<BWD>(in, m, len, wt, r, out, sms, st);
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// int8 matrix [rows, cols] with rows `ld` bytes apart, box [brows, 128 bytes].
bool make_map_i8(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t brows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {ld};
    cuuint32_t box[2] = {128, brows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The plan of one call's product: CTA pairs on 256 x 256 tiles when these fill
// the machine, else split CTAs on token tiles of nt, with the reduction in
// nsplit parts.
struct I8Plan {
    bool pair;
    I8SplitShape sh;             // split CTAs
    int nsplit;
};

I8Plan plan_i8(int m, int64_t out, int64_t red, int sms) {
    I8Plan pl{};
    const int64_t blocks = cdiv(red, 128);
    if (m > 128 && cdiv(out, kI8Tile) * cdiv(m, kI8Tile) >= sms / 2) {
        pl.pair = true;
        return pl;
    }
    // token tiles of at most 128 where one wave of two CTAs per SM holds them, else of at
    // most 256 (1024 tokens x 4096 x 4096 at rank 16: 38 us with tiles of 128, 45 with 256,
    // whose epilogue no other CTA of the SM hides); smaller ones, down to 32, where the
    // output features and the parts of the reduction leave SMs idle (3913 tokens x 78 x 64,
    // rank 64, took 82 us on 16 CTAs of 256 tokens)
    const int64_t rtiles = cdiv(out, 128), smax = std::min<int64_t>(kI8MaxSplit, std::max<int64_t>(1, blocks / 4));
    const int64_t widest = rtiles * cdiv(m, 128) <= 2 * sms ? 128 : 256;
    const int64_t ttiles =
        std::max<int64_t>(cdiv(m, widest), std::min<int64_t>(cdiv(m, 32), sms / (rtiles * smax)));
    pl.sh.nt = static_cast<int>(round_up(static_cast<size_t>(cdiv(m, ttiles)), 16));
    // two CTAs per SM while their rings hold three blocks each
    const int per_sm = pl.sh.nt <= 128 ? 2 : 1;
    const int64_t tiles = rtiles * cdiv(m, pl.sh.nt), want = std::max<int64_t>(1, per_sm * sms / tiles);
    pl.nsplit = parts_that_fit(std::min<int64_t>(want, smax), tiles, per_sm, sms);
    pl.sh.tok = static_cast<int>(cdiv(pl.sh.nt, pl.nsplit));
    return pl;
}

// The ring of a split CTA: as many blocks as its share of the SM's shared
// memory holds beside the factors of its tokens (rank rounded to rp), at least 2.
I8SplitShape split_shape(const I8Plan& pl, int64_t red, int rp) {
    I8SplitShape sh = pl.sh;
    const int64_t budget = (sh.nt <= 128 ? 106 : 210) * 1024 - int64_t(sh.tok) * rp * 4 - sh.nt * 4;
    const int64_t blocks = std::max<int64_t>(2, cdiv(cdiv(red, 128), pl.nsplit));
    sh.stages = static_cast<int>(std::min<int64_t>({kI8SplitMaxStages, blocks, std::max<int64_t>(2, budget / sh.stage_bytes())}));
    return sh;
}

// Codes and scales of the tokens in a call's workspace.
struct I8Space {
    int64_t ld;          // bytes of a code row, a multiple of 16
    size_t scale_at, bytes;
};

I8Space i8_space(int m, int64_t red) {
    I8Space t;
    t.ld = static_cast<int64_t>(round_up(static_cast<size_t>(red), 16));
    t.scale_at = round_up(static_cast<size_t>(m) * static_cast<size_t>(t.ld), 256);
    t.bytes = t.scale_at + round_up(static_cast<size_t>(m) * sizeof(float), 256);
    return t;
}

struct I8Job {
    const lbq_i8weight* w;
    const void* tokens;    // bf16 [m, red]
    const float* chan;     // their channel scales (backward)
    const void* factor;    // the adapter's factor that multiplies the tokens
    float* saved;          // their product
    int8_t* codes;         // of the tokens, in the workspace
    float* scale;
    int64_t ld;
    I8Params p;
};

template <bool TRANS, int RP>
lbq_status launch_i8_split(const I8Job& j, const I8Plan& pl, cudaStream_t st) {
    CUtensorMap tmW, tmX;
    if (!make_map_i8(&tmW, j.w->codes, j.w->n, j.w->k, j.w->k, 128) ||
        !make_map_i8(&tmX, j.codes, j.p.m, j.p.red, j.ld, pl.sh.nt))
        return LBQ_ECUDA;
    const I8SplitShape sh = split_shape(pl, j.p.red, RP);
    const dim3 grid(static_cast<unsigned>(cdiv(j.p.out, 128)), static_cast<unsigned>(cdiv(j.p.m, sh.nt)),
                    static_cast<unsigned>(pl.nsplit));
    return launch_overlapped<i8_split_kernel<TRANS, RP>>(grid, kI8SplitThreads, sh.bytes(RP),
                                                         dim3(1, 1, static_cast<unsigned>(pl.nsplit)), st, tmW, tmX, j.p, sh);
}

template <bool TRANS, int RP>
lbq_status launch_i8_pair(const I8Job& j, int sms, cudaStream_t st) {
    CUtensorMap tmW, tmX;
    if (!make_map_i8(&tmW, j.w->codes, j.w->n, j.w->k, j.w->k, 128) ||
        !make_map_i8(&tmX, j.codes, j.p.m, j.p.red, j.ld, 128))
        return LBQ_ECUDA;
    const int64_t tiles = cdiv(j.p.out, kI8Tile) * cdiv(j.p.m, kI8Tile);
    const unsigned pairs = static_cast<unsigned>(std::min<int64_t>(tiles, std::max(1, sms / 2)));
    return launch_overlapped<i8_pair_kernel<TRANS, RP>>(dim3(2 * pairs), kI8PairThreads, I8PairCfg<RP>::kBytes,
                                                        dim3(2, 1, 1), st, tmW, tmX, j.p);
}

// The adapter's product, the tokens' codes, the product.
template <bool TRANS, int RP>
lbq_status run_i8_product(const I8Job& j, const I8Plan& pl, int sms, cudaStream_t st) {
    lbq_status s = LBQ_OK;
    if (RP > 0) s = run_i8_factor<TRANS>(j.tokens, j.p.m, j.p.red, j.factor, j.p.rank, j.saved, sms, st);
    if (s == LBQ_OK)
        s = run_i8_quantize<kSrcBf16, TRANS, (RP > 0)>(j.tokens, j.p.m, j.p.red, j.chan, j.codes, j.ld, j.scale, sms, st);
    if (s != LBQ_OK) return s;
    return pl.pair ? launch_i8_pair<TRANS, RP>(j, sms, st) : launch_i8_split<TRANS, RP>(j, pl, st);
}

// One call: forward (TRANS false, in = X) or input gradient (in = dY).  A and B
// are the adapter's factors, saved its product with the tokens.
template <bool TRANS>
lbq_status run_i8_linear(const void* in, int m, const lbq_i8weight* q, const void* A, const void* B, int rank, float s,
                         float* out, float* saved, void* ws, const I8Space& at, int sms, cudaStream_t st) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    I8Job j{};
    j.w = q;
    j.tokens = in;
    j.chan = TRANS ? q->scale : nullptr;
    j.factor = TRANS ? B : A;
    j.saved = saved;
    j.codes = reinterpret_cast<int8_t*>(w);
    j.scale = reinterpret_cast<float*>(w + at.scale_at);
    j.ld = at.ld;
    j.p.m = m;
    j.p.out = TRANS ? q->k : q->n;
    j.p.red = TRANS ? q->n : q->k;
    j.p.row_scale = j.scale;
    j.p.out_scale = TRANS ? nullptr : q->scale;
    j.p.rank = rank;
    j.p.s = s;
    j.p.T = saved;
    j.p.P = static_cast<const uint16_t*>(TRANS ? A : B);
    j.p.pj = TRANS ? 1 : rank;
    j.p.pu = TRANS ? q->k : 1;
    j.p.Y = out;
    const I8Plan pl = plan_i8(m, j.p.out, j.p.red, sms);
    if (rank == 0) return run_i8_product<TRANS, 0>(j, pl, sms, st);
    if (rank <= 16) return run_i8_product<TRANS, 16>(j, pl, sms, st);
    return run_i8_product<TRANS, 64>(j, pl, sms, st);
}
