// i8_host.cuh -- host side of the 8-bit integer products: argument checks, the
// choice of kernel and split, tensor maps and launches.  Included by lbq.cu
// inside its anonymous namespace.

// Launch with optional cluster size and programmatic stream serialisation
// (the kernel waits with griddepcontrol.wait before it reads what the kernel
// before it wrote).
template <typename... KArgs, typename... Args>
lbq_status launch_overlapped(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, dim3 cluster, cudaStream_t st,
                             Args... args) {
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
        (void)cudaGetLastError();
        return LBQ_ECUDA;
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
    if (cudaLaunchKernelEx(&cfg, kern, KArgs(args)...) != cudaSuccess) {
        (void)cudaGetLastError();
        return LBQ_ECUDA;
    }
    return last_launch();
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
                           float* scale, cudaStream_t st) {
    const int64_t nvec = len / 8;
    auto go = [&](auto kern, int threads) {
        return launch_overlapped(kern, dim3(static_cast<unsigned>(rows)), threads, 0, dim3(1, 1, 1), st, in, len, chan,
                                 codes, ldc, scale);
    };
    // the fewest threads that hold the row in registers, up to 64 bytes each
    if (nvec <= 256) return go(i8_quantize_rows_kernel<SRC, SCALED, BESIDE, 1, 256>, 256);
    if (nvec <= 512) return go(i8_quantize_rows_kernel<SRC, SCALED, BESIDE, 2, 256>, 256);
    if (nvec <= 1024) return go(i8_quantize_rows_kernel<SRC, SCALED, BESIDE, 4, 256>, 256);
    if (nvec <= 2048) return go(i8_quantize_rows_kernel<SRC, SCALED, BESIDE, 4, 512>, 512);
    if (nvec <= 4096) return go(i8_quantize_rows_kernel<SRC, SCALED, BESIDE, 4, 1024>, 1024);
    return go(i8_quantize_rows_kernel<SRC, SCALED, BESIDE, 0, 1024>, 1024);
}

template <bool COL, int MT, int R8>
lbq_status launch_i8_adapter(const void* in, int64_t m, int64_t len, const void* wt, int r, float* out, int sms,
                             cudaStream_t st) {
    // parts enough for two CTAs per SM
    const int64_t groups = cdiv(m, MT), chunks = cdiv(len, kAdChunk);
    const int64_t parts = std::min<int64_t>({kAdMaxParts, chunks, std::max<int64_t>(1, 2 * sms / groups)});
    return launch_overlapped(i8_adapter_kernel<COL, MT, R8>, dim3(static_cast<unsigned>(groups), static_cast<unsigned>(parts)),
                             kAdThreads, AdapterSmem<MT, R8>::kBytes, dim3(1, static_cast<unsigned>(parts), 1), st,
                             static_cast<const uint16_t*>(in), m, static_cast<int>(len), static_cast<const uint16_t*>(wt), r,
                             out);
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
    const int64_t parts = std::min<int64_t>({kAdMaxParts, blocks, std::max<int64_t>(1, sms / groups)});
    return launch_overlapped(i8_adapter_tc_kernel<COL, NR>, dim3(static_cast<unsigned>(groups), static_cast<unsigned>(parts)),
                             kAdTcThreads, AdapterTcSmem<NR>::kBytes, dim3(1, static_cast<unsigned>(parts), 1), st, tmX, tmW,
                             static_cast<int>(m), static_cast<int>(len), r, out);
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

// Codes and scales of the tokens and, with an adapter, its product `out`.
template <bool BWD>
lbq_status run_i8_tokens(const void* in, int64_t m, int64_t len, const float* chan, const void* wt, int r, int8_t* codes,
                         int64_t ldc, float* scale, float* out, int sms, cudaStream_t st) {
    if (r == 0) return run_i8_quantize<kSrcBf16, BWD, false>(in, m, len, chan, codes, ldc, scale, st);
    const lbq_status s = m <= 16                 ? run_i8_adapter<BWD, 16>(in, m, len, wt, r, out, sms, st)
                         : !BWD || r % 8 == 0 ? run_i8_adapter_tc<BWD>(in, m, len, wt, r, out, sms, st)
                                              : run_i8_adapter<BWD, 64>(in, m, len, wt, r, out, sms, st);
    if (s != LBQ_OK) return s;
    return run_i8_quantize<kSrcBf16, BWD, true>(in, m, len, chan, codes, ldc, scale, st);
}

// Codes and scales of the tokens in a call's workspace.
struct I8Tokens {
    int64_t ld;          // bytes of a code row, a multiple of 16
    size_t scale_at;     // offset of the scales
    size_t bytes;
};

I8Tokens i8_tokens(int m, int64_t len) {
    I8Tokens t;
    t.ld = static_cast<int64_t>(round_up(static_cast<size_t>(len), 16));
    t.scale_at = round_up(static_cast<size_t>(m) * static_cast<size_t>(t.ld), 256);
    t.bytes = t.scale_at + round_up(static_cast<size_t>(m) * sizeof(float), 256);
    return t;
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

struct I8Job {
    const lbq_i8weight* w;
    const int8_t* codes;   // tokens
    int64_t ld;
    I8Params p;
};

template <int NT, bool TRANS, int RP>
lbq_status launch_i8_split(const I8Job& j, int nsplit, cudaStream_t st) {
    CUtensorMap tmW, tmX;
    if (!make_map_i8(&tmW, j.w->codes, j.w->n, j.w->k, j.w->k, 128) ||
        !make_map_i8(&tmX, j.codes, j.p.m, j.p.red, j.ld, NT))
        return LBQ_ECUDA;
    const dim3 grid(static_cast<unsigned>(cdiv(j.p.out, 128)), static_cast<unsigned>(cdiv(j.p.m, NT)),
                    static_cast<unsigned>(nsplit));
    return launch_overlapped(i8_split_kernel<NT, TRANS, RP>, grid, kI8SplitThreads, I8SplitCfg<NT>::kBytes,
                             dim3(1, 1, static_cast<unsigned>(nsplit)), st, tmW, tmX, j.p);
}

template <int NT, bool TRANS, int RP>
lbq_status launch_i8_pair(const I8Job& j, int sms, cudaStream_t st) {
    CUtensorMap tmW, tmX;
    if (!make_map_i8(&tmW, j.w->codes, j.w->n, j.w->k, j.w->k, 128) ||
        !make_map_i8(&tmX, j.codes, j.p.m, j.p.red, j.ld, NT / 2))
        return LBQ_ECUDA;
    const int64_t tiles = cdiv(j.p.out, 256) * cdiv(j.p.m, NT);
    const unsigned pairs = static_cast<unsigned>(std::min<int64_t>(tiles, std::max(1, sms / 2)));
    return launch_overlapped(i8_pair_kernel<NT, TRANS, RP>, dim3(2 * pairs), kI8PairThreads, (I8PairCfg<NT, RP>::kBytes),
                             dim3(2, 1, 1), st, tmW, tmX, j.p);
}

struct I8Plan {
    int nt;        // tokens of a tile
    bool pair;     // CTA pairs, else split CTAs
    int nsplit;    // parts of the reduction (split CTAs)
};

I8Plan plan_i8(int m, int64_t out, int64_t red, int sms) {
    I8Plan pl{};
    pl.nt = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
    pl.nsplit = 1;
    if (m > 128 && cdiv(out, 256) * cdiv(m, 256) >= sms / 2) {
        pl.pair = true;
        pl.nt = 256;
        return pl;
    }
    const int64_t tiles = cdiv(out, 128) * cdiv(m, pl.nt), blocks = cdiv(red, 128);
    const int64_t want = std::max<int64_t>(1, 2 * sms / tiles);
    pl.nsplit = static_cast<int>(std::min<int64_t>({want, kI8MaxSplit, std::max<int64_t>(1, blocks / 4)}));
    return pl;
}

template <bool TRANS, int RP>
lbq_status run_i8_product_rp(const I8Job& j, int sms, cudaStream_t st) {
    const I8Plan pl = plan_i8(j.p.m, j.p.out, j.p.red, sms);
    if (pl.pair) return launch_i8_pair<256, TRANS, RP>(j, sms, st);
    if (cdiv(j.p.m, pl.nt) > 65535) return LBQ_EUNSUPPORTED;
    switch (pl.nt) {
        case 16: return launch_i8_split<16, TRANS, RP>(j, pl.nsplit, st);
        case 32: return launch_i8_split<32, TRANS, RP>(j, pl.nsplit, st);
        case 64: return launch_i8_split<64, TRANS, RP>(j, pl.nsplit, st);
        default: return launch_i8_split<128, TRANS, RP>(j, pl.nsplit, st);
    }
}

template <bool TRANS>
lbq_status run_i8_product(const I8Job& j, int sms, cudaStream_t st) {
    if (j.p.rank == 0) return run_i8_product_rp<TRANS, 0>(j, sms, st);
    if (j.p.rank <= 16) return run_i8_product_rp<TRANS, 16>(j, sms, st);
    return run_i8_product_rp<TRANS, 64>(j, sms, st);
}
