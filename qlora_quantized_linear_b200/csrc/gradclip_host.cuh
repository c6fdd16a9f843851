// gradclip_host.cuh -- host side of the gradient norm and clipping: argument
// checks, the tensor tables and the launches.  Included by lbq.cu inside its
// anonymous namespace.

constexpr size_t kClipHeader = 256;       // the grid barrier's two words, then the total at byte 64

int clip_launches(int count) { return static_cast<int>(cdiv(count, kClipTable)); }

size_t clip_workspace(int count) {
    return kClipHeader + static_cast<size_t>(clip_launches(count)) * kClipMaxCtas * sizeof(double);
}

struct ByteRange {
    uintptr_t lo, hi;
    bool operator<(const ByteRange& o) const { return lo < o.lo; }
};

// No output may overlap another output or another tensor's input: the kernels
// read and write them in no stated order.  (An output may be its own input.)
lbq_status check_grad_outputs(const lbq_grad* grads, int count) {
    std::vector<ByteRange> outs;
    try {
        outs.reserve(count);
    } catch (...) {
        return LBQ_ECUDA;
    }
    auto bytes = [](const lbq_grad& g) { return static_cast<uintptr_t>(g.numel) * (g.dtype == LBQ_F32 ? 4u : 2u); };
    for (int i = 0; i < count; ++i) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(grads[i].out);
        if (grads[i].numel > 0) outs.push_back(ByteRange{lo, lo + bytes(grads[i])});
    }
    if (!std::is_sorted(outs.begin(), outs.end())) std::sort(outs.begin(), outs.end());
    for (size_t i = 1; i < outs.size(); ++i)
        if (outs[i].lo < outs[i - 1].hi) return LBQ_EINVAL;
    for (int i = 0; i < count; ++i) {
        if (grads[i].numel == 0 || grads[i].g == grads[i].out) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(grads[i].g), hi = lo + bytes(grads[i]);
        // the last output that starts before this input ends
        auto it = std::lower_bound(outs.begin(), outs.end(), ByteRange{hi, hi});
        if (it != outs.begin() && (--it)->hi > lo) return LBQ_EINVAL;
    }
    return LBQ_OK;
}

lbq_status check_grads(const lbq_grad* grads, int count, bool clip) {
    if (!grads || count < 1) return LBQ_EINVAL;
    for (int i = 0; i < count; ++i) {
        const lbq_grad& g = grads[i];
        if (g.dtype != LBQ_F32 && g.dtype != LBQ_BF16 && g.dtype != LBQ_F16) return LBQ_EUNSUPPORTED;
        if (g.numel < 0 || g.numel > (int64_t(1) << 40)) return LBQ_EINVAL;
        if (g.numel == 0) continue;
        if (!g.g || (clip && !g.out)) return LBQ_EINVAL;
        const uintptr_t mask = g.dtype == LBQ_F32 ? 3u : 1u;
        if ((reinterpret_cast<uintptr_t>(g.g) & mask) || (clip && (reinterpret_cast<uintptr_t>(g.out) & mask)))
            return LBQ_EALIGN;
    }
    return clip ? check_grad_outputs(grads, count) : LBQ_OK;
}

template <int MODE, int CAP>
lbq_status launch_clip(const lbq_grad* grads, int count, const ClipWork& wk, int sms, cudaStream_t st) {
    ClipTable<CAP> tab;
    tab.count = 0;
    uint64_t chunks = 0;
    for (int i = 0; i < count; ++i) {
        const lbq_grad& g = grads[i];
        if (g.numel == 0) continue;
        const int64_t size = g.dtype == LBQ_F32 ? 4 : 2;
        const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(g.g) & 15u) / size;
        ClipEntry& e = tab.e[tab.count++];
        e.g = static_cast<const uint8_t*>(g.g) - lead * size;
        e.out = static_cast<uint8_t*>(g.out) - (g.out ? lead * size : 0);
        e.end = lead + g.numel;
        e.chunk0 = static_cast<uint32_t>(chunks);
        e.type = static_cast<uint16_t>(g.dtype);
        e.lead = static_cast<uint16_t>(lead);
        chunks += static_cast<uint64_t>(cdiv(e.end * size, kClipChunk));
    }
    if (chunks >= (uint64_t(1) << 31)) return LBQ_EUNSUPPORTED;
    tab.chunks = static_cast<uint32_t>(chunks);
    // the first tensor of each CTA's range (the last that starts at or before the range's first chunk)
    const int grid = std::min(sms, kClipMaxCtas);
    for (int b = 0, t = 0; b <= grid; ++b) {
        const uint64_t c = chunks * b / grid;
        while (t + 1 < tab.count && tab.e[t + 1].chunk0 <= c) ++t;
        tab.first[b] = static_cast<uint16_t>(t);
    }
    auto kern = grad_clip_kernel<MODE, CAP>;
    constexpr size_t smem = clip_smem_bytes<CAP>();
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
                        cudaSuccess) {
        (void)cudaGetLastError();
        return LBQ_ECUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kClipThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = MODE == kClipFused ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, tab, wk) != cudaSuccess) {
        (void)cudaGetLastError();
        return LBQ_ECUDA;
    }
    return last_launch();
}

lbq_status run_clip(const lbq_grad* grads, int count, bool clip, float max_norm, float* norm, void* ws,
                    cudaStream_t st) {
    const int sms = sm_count(), launches = clip_launches(count);
    ClipWork wk{};
    wk.bar = static_cast<uint32_t*>(ws);
    wk.total = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + 64);
    wk.part = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + kClipHeader);
    wk.norm = norm;
    wk.max_norm = max_norm;
    const int grid = std::min(sms, kClipMaxCtas);
    wk.nparts = launches * grid;
    if (launches == 1) {
        // a small table where it suffices: the launch carries the whole of it
        if (count <= 64)
            return clip ? launch_clip<kClipFused, 64>(grads, count, wk, sms, st)
                        : launch_clip<kClipSumLast, 64>(grads, count, wk, sms, st);
        if (count <= 512)
            return clip ? launch_clip<kClipFused, 512>(grads, count, wk, sms, st)
                        : launch_clip<kClipSumLast, 512>(grads, count, wk, sms, st);
        return clip ? launch_clip<kClipFused, kClipTable>(grads, count, wk, sms, st)
                    : launch_clip<kClipSumLast, kClipTable>(grads, count, wk, sms, st);
    }
    // more tensors than a launch describes: all sums, then all products
    for (int l = 0; l < launches; ++l) {
        wk.part0 = l * grid;
        const int c = std::min(kClipTable, count - l * kClipTable);
        const lbq_status s = l + 1 < launches ? launch_clip<kClipSum, kClipTable>(grads + l * kClipTable, c, wk, sms, st)
                                              : launch_clip<kClipSumLast, kClipTable>(grads + l * kClipTable, c, wk, sms, st);
        if (s != LBQ_OK) return s;
    }
    for (int l = 0; clip && l < launches; ++l) {
        const lbq_status s = launch_clip<kClipScale, kClipTable>(grads + l * kClipTable,
                                                                 std::min(kClipTable, count - l * kClipTable), wk, sms, st);
        if (s != LBQ_OK) return s;
    }
    return LBQ_OK;
}
