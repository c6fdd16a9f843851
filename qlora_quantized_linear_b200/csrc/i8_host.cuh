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
template <int SRC, bool SCALED>
lbq_status run_i8_quantize(const void* in, int64_t rows, int64_t len, const float* chan, int8_t* codes, int64_t ldc,
                           float* scale, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(rows)), one(1, 1, 1);
    const int64_t nvec = len / 8;
    // the fewest threads that hold the row in registers with up to 32 values each
    if (nvec <= 256)
        return launch_overlapped(i8_quantize_rows_kernel<SRC, SCALED, 1, 256>, grid, 256, 0, one, st, in, len, chan,
                                 codes, ldc, scale);
    if (nvec <= 512)
        return launch_overlapped(i8_quantize_rows_kernel<SRC, SCALED, 2, 256>, grid, 256, 0, one, st, in, len, chan,
                                 codes, ldc, scale);
    if (nvec <= 1024)
        return launch_overlapped(i8_quantize_rows_kernel<SRC, SCALED, 4, 256>, grid, 256, 0, one, st, in, len, chan,
                                 codes, ldc, scale);
    if (nvec <= 2048)
        return launch_overlapped(i8_quantize_rows_kernel<SRC, SCALED, 4, 512>, grid, 512, 0, one, st, in, len, chan,
                                 codes, ldc, scale);
    if (nvec <= 4096)
        return launch_overlapped(i8_quantize_rows_kernel<SRC, SCALED, 4, 1024>, grid, 1024, 0, one, st, in, len, chan,
                                 codes, ldc, scale);
    return launch_overlapped(i8_quantize_rows_kernel<SRC, SCALED, 0, 1024>, grid, 1024, 0, one, st, in, len, chan,
                             codes, ldc, scale);
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
    return launch_overlapped(i8_pair_kernel<NT, TRANS, RP>, dim3(2 * pairs), kI8PairThreads, I8PairCfg<NT>::kBytes,
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
