// tree_api.cuh - C entry points of the draft-tree calls (part of oasis.cu).

namespace {

// Launch attributes of a kernel set once per device instead of on every call.
struct OncePerDevice {
    std::mutex mu;
    uint64_t done = 0;
    template <class F>
    int operator()(F&& f) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 64 && (done >> dev & 1)) return OASIS_OK;
        if (int rc = f()) return rc;
        if (dev < 64) done |= 1ull << dev;
        return OASIS_OK;
    }
};

int check_tree(const oasis_dims* dp, int32_t n_tree, Dims* d) {
    if (int rc = validate(dp, d)) return rc;
    if (n_tree < 1 || n_tree > oasis::kMaxTree)
        return fail(OASIS_EINVAL, "n_tree must be in [1, 64] (got %d)", n_tree);
    return OASIS_OK;
}

// The tree's keys or values: bf16 [B*Hkv][T][128] as a 3-D tensor, boxes of
// 64 columns x the nodes padded to whole slots; rows past T read as zeros.
int make_map_tree(CUtensorMap* m, const void* base, unsigned long long units, int T, const char* name) {
    auto fn = encode_fn();
    if (fn == nullptr) return fail(OASIS_ECUDA, "cuTensorMapEncodeTiled unavailable");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(oasis::kHeadDim), static_cast<cuuint64_t>(T),
                                static_cast<cuuint64_t>(units)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(oasis::kRowBytes),
                                   static_cast<cuuint64_t>(oasis::kRowBytes) * T};
    const int t16 = (T + oasis::kBlockTokens - 1) / oasis::kBlockTokens * oasis::kBlockTokens;
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(t16), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(OASIS_ECUDA, "cuTensorMapEncodeTiled(%s) failed: %d", name, static_cast<int>(r));
    return OASIS_OK;
}

// Work of a tree attention call: items of up to two row tiles (128 query rows
// each, whole nodes), KV tiles a unit (8 slots each, and the tree's own), and
// the equal stretch of all items' KV tiles that a CTA takes.  An SM that the
// gather occupies cannot hold an attention CTA beside it (as in
// oasis_sparse_attn), so the gather's SMs are left free.
struct TreeWork {
    int nt, pairs, tpu, per, total, ctas, grid_max;
};

TreeWork tree_work(const Dims& d, int T) {
    TreeWork w;
    w.nt = std::min(T, oasis::kTaRows / d.G());
    const int tiles = (T + w.nt - 1) / w.nt;
    w.pairs = (tiles + 1) / 2;
    w.tpu = (d.K + oasis::kAttnTileSlots - 1) / oasis::kAttnTileSlots + 1;
    const long long total = static_cast<long long>(d.B) * d.Hkv * w.pairs * w.tpu;
    w.total = static_cast<int>(total);           // <= 65535 units x 64 pairs x 129 tiles: below 2^31 (checked by the caller)
    w.grid_max = std::max(1, sm_count() - oasis::kPrefetchCtas);
    w.per = static_cast<int>((total + w.grid_max - 1) / w.grid_max);
    w.per = std::max(w.per, std::min(w.tpu, 2));
    // whole items where that makes no CTA's share much longer: a split item costs its parts' trip through the
    // workspace and the joining, about four tiles' time
    const int whole = (w.per + w.tpu - 1) / w.tpu * w.tpu;
    if (whole <= w.per + 4) w.per = whole;
    w.ctas = static_cast<int>((total + w.per - 1) / w.per);
    return w;
}

// Workspace: the parts' outputs and log2-sum-exps, two places a CTA.
struct TreeWs {
    size_t o, lse, total;
};

TreeWs tree_ws(const Dims& d, const TreeWork& w) {
    TreeWs s;
    const size_t rows = static_cast<size_t>(w.grid_max) * 2 * 256;
    s.o = 0;
    s.lse = align256(rows * oasis::kHeadDim * sizeof(float));
    s.total = align256(s.lse + rows * sizeof(float));
    return s;
}

int check_tree_heads(const Dims& d) {
    if (d.G() > 64) return fail(OASIS_EINVAL, "n_q_heads / n_kv_heads must be <= 64 (got %d)", d.G());
    return OASIS_OK;
}

}  // namespace

extern "C" {

int oasis_tree_layout(const oasis_dims* dp, int32_t n_tree, const int32_t* parent, const int32_t* n_nodes,
                      const int32_t* ctx_len, uint64_t* mask, int32_t* pos, void* stream) {
    Dims d;
    if (int rc = check_tree(dp, n_tree, &d)) return rc;
    if (int rc = check_ptr(parent, "parent")) return rc;
    if (int rc = check_ptr(n_nodes, "n_nodes", true)) return rc;
    if (int rc = check_ptr(ctx_len, "ctx_len")) return rc;
    if (int rc = check_ptr(mask, "mask")) return rc;
    if (int rc = check_ptr(pos, "pos")) return rc;
    static OncePerDevice once;
    if (int rc = once([] { return carveout(oasis::tree_layout_kernel, "tree_layout carve-out"); })) return rc;
    const unsigned grid = (d.B + oasis::kLayoutTrees - 1) / oasis::kLayoutTrees;
    oasis::tree_layout_kernel<<<grid, oasis::kLayoutTrees * oasis::kMaxTree, 0, static_cast<cudaStream_t>(stream)>>>(
        d.B, n_tree, parent, n_nodes, ctx_len, mask, pos);
    return check_launch("tree_layout launch");
}

int oasis_qk_norm_rope(const oasis_dims* dp, int32_t n_tok, const void* qkv, size_t row_stride, const void* wq,
                       const void* wk, float eps, const float* inv_freq, const int32_t* pos, void* q, void* k, void* v,
                       void* stream) {
    Dims d;
    if (int rc = validate(dp, &d)) return rc;
    if (n_tok < 1) return fail(OASIS_EINVAL, "n_tok must be >= 1 (got %d)", n_tok);
    if (int rc = check_ptr(qkv, "qkv")) return rc;
    if (int rc = check_ptr(wq, "wq", true)) return rc;
    if (int rc = check_ptr(wk, "wk", true)) return rc;
    if (int rc = check_ptr(inv_freq, "inv_freq")) return rc;
    if (int rc = check_ptr(pos, "pos")) return rc;
    if (int rc = check_ptr(q, "q")) return rc;
    if (int rc = check_ptr(k, "k")) return rc;
    if (int rc = check_ptr(v, "v")) return rc;
    const int heads = d.Hq + 2 * d.Hkv;
    if (row_stride < static_cast<size_t>(heads) * oasis::kHeadDim || row_stride % 8 != 0 || row_stride > (size_t(1) << 40))
        return fail(OASIS_EINVAL, "row_stride must be a multiple of 8 and >= (Hq + 2 Hkv) * 128 (got %zu)", row_stride);
    if (!(eps >= 0.f) || !(eps < 3.0e38f)) return fail(OASIS_EINVAL, "eps must be a finite float >= 0");
    static OncePerDevice once;
    if (int rc = once([] { return carveout(oasis::qk_norm_rope_kernel, "qk_norm_rope carve-out"); })) return rc;
    // Warps a token: one while there are enough tokens to fill the SMs (its
    // angles are then made once), more when there are few.
    const long long tokens = static_cast<long long>(d.B) * n_tok;
    const int steps = (heads + oasis::kRopeStep - 1) / oasis::kRopeStep;
    const long long fill = 32ll * sm_count();
    const int split = static_cast<int>(std::min<long long>(steps, std::max<long long>(1, fill / tokens)));
    const long long grid = (tokens * split + oasis::kRopeWarps - 1) / oasis::kRopeWarps;
    if (grid > 0x7FFFFFFFll) return fail(OASIS_EINVAL, "too many tokens");
    oasis::qk_norm_rope_kernel<<<static_cast<unsigned>(grid), oasis::kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        d, n_tok, split, static_cast<const uint16_t*>(qkv), static_cast<long long>(row_stride), static_cast<const uint16_t*>(wq),
        static_cast<const uint16_t*>(wk), eps, inv_freq, pos, static_cast<uint16_t*>(q), static_cast<uint16_t*>(k),
        static_cast<uint16_t*>(v));
    return check_launch("qk_norm_rope launch");
}

size_t oasis_tree_workspace_bytes(const oasis_dims* dp, int32_t n_tree) {
    Dims d;
    if (check_tree(dp, n_tree, &d) != OASIS_OK || check_tree_heads(d) != OASIS_OK) return 0;
    return tree_ws(d, tree_work(d, n_tree)).total;
}

int oasis_tree_attn(const oasis_dims* dp, int32_t n_tree, const void* q, const void* pool, const int32_t* slot_table,
                    const int32_t* ctx_len, const void* k_tree, const void* v_tree, const uint64_t* mask, float scale,
                    void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    Dims d;
    if (int rc = check_tree(dp, n_tree, &d)) return rc;
    if (int rc = check_tree_heads(d)) return rc;
    if (int rc = check_ptr(q, "q")) return rc;
    if (int rc = check_ptr(pool, "pool")) return rc;
    if (int rc = check_ptr(slot_table, "slot_table")) return rc;
    if (int rc = check_ptr(ctx_len, "ctx_len")) return rc;
    if (int rc = check_ptr(k_tree, "k_tree")) return rc;
    if (int rc = check_ptr(v_tree, "v_tree")) return rc;
    if (int rc = check_ptr(mask, "mask")) return rc;
    if (int rc = check_ptr(out, "out")) return rc;
    if (int rc = check_ptr(lse, "lse")) return rc;
    if (int rc = check_ptr(ws, "ws")) return rc;
    if (!(scale > 0.f) || !(scale < 3.0e38f)) return fail(OASIS_EINVAL, "scale must be a positive finite float");
    const TreeWork w = tree_work(d, n_tree);
    if (static_cast<long long>(d.B) * d.Hkv * w.pairs * w.tpu > 0x3FFFFFFFll) return fail(OASIS_EINVAL, "too many rows");
    const TreeWs ly = tree_ws(d, w);
    if (ws_bytes < ly.total) return fail(OASIS_EINVAL, "workspace too small: %zu < %zu", ws_bytes, ly.total);
    CUtensorMap tk, tv, tq, ttk, ttv;
    const unsigned long long units = static_cast<unsigned long long>(d.B) * d.Hkv;
    if (int rc = make_map_pool(&tk, pool, units * d.K, "pool keys")) return rc;
    if (int rc = make_map_pool(&tv, static_cast<const uint8_t*>(pool) + oasis::kBlockBytes / 2, units * d.K, "pool values"))
        return rc;
    if (int rc = make_map_tree(&ttk, k_tree, units, n_tree, "tree keys")) return rc;
    if (int rc = make_map_tree(&ttv, v_tree, units, n_tree, "tree values")) return rc;
    Dims dq = d;
    dq.Qn = n_tree;
    if (int rc = make_map_q(&tq, q, dq, w.nt)) return rc;
    static OncePerDevice once;
    if (int rc = once([] {
            if (int rc = carveout(oasis::tree_join_kernel, "tree_join carve-out")) return rc;
            return set_smem(oasis::tree_attn_kernel, oasis::kTaSmem, "tree_attn smem");
        }))
        return rc;
    uint8_t* base = static_cast<uint8_t*>(ws);
    oasis::TreeAttnArgs a;
    a.slot_table = slot_table;
    a.ctx_len = ctx_len;
    a.mask = mask;
    a.v_tree = static_cast<const uint16_t*>(v_tree);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.ws_o = reinterpret_cast<float*>(base + ly.o);
    a.ws_lse = reinterpret_cast<float*>(base + ly.lse);
    a.scale_log2 = scale * 1.4426950408889634f;
    a.T = n_tree;
    a.nt = w.nt;
    a.units = d.B * d.Hkv;
    a.tpu = w.tpu;
    a.per = w.per;
    a.total = w.total;
    oasis::tree_attn_kernel<<<static_cast<unsigned>(w.ctas), oasis::kTaThreads, oasis::kTaSmem,
                              static_cast<cudaStream_t>(stream)>>>(tk, tv, tq, ttk, ttv, d, a);
    if (int rc = check_launch("tree_attn launch")) return rc;
    if (w.per % w.tpu == 0) return OASIS_OK;     // whole items
    const unsigned rows = static_cast<unsigned>(d.B) * n_tree * d.Hq;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((rows + oasis::kTjWarps - 1) / oasis::kTjWarps);
    cfg.blockDim = dim3(32 * oasis::kTjWarps);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, oasis::tree_join_kernel, d, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail(e, "tree_join launch");
    }
    return check_launch("tree_join launch");
}

int oasis_verify_tree(const oasis_dims* dp, int32_t n_tree, int32_t vocab, const float* probs, const float* draft_probs,
                      size_t row_stride, const int32_t* tokens, const int32_t* parent, const int32_t* n_nodes,
                      const float* u_accept, const float* u_sample, int32_t* path, int32_t* n_accept,
                      int32_t* next_token, void* stream) {
    Dims d;
    if (int rc = check_tree(dp, n_tree, &d)) return rc;
    if (vocab < 1 || vocab > (1 << 30)) return fail(OASIS_EINVAL, "vocab must be in [1, 2^30] (got %d)", vocab);
    if (row_stride < static_cast<size_t>(vocab) || row_stride > (size_t(1) << 40))
        return fail(OASIS_EINVAL, "row_stride must be >= vocab (got %zu)", row_stride);
    if (int rc = check_ptr(probs, "probs")) return rc;
    if (int rc = check_ptr(draft_probs, "draft_probs", true)) return rc;
    if (int rc = check_ptr(tokens, "tokens")) return rc;
    if (int rc = check_ptr(parent, "parent")) return rc;
    if (int rc = check_ptr(n_nodes, "n_nodes", true)) return rc;
    if (int rc = check_ptr(u_accept, "u_accept")) return rc;
    if (int rc = check_ptr(u_sample, "u_sample")) return rc;
    if (int rc = check_ptr(path, "path")) return rc;
    if (int rc = check_ptr(n_accept, "n_accept")) return rc;
    if (int rc = check_ptr(next_token, "next_token")) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(oasis::kVerThreads);
    cfg.dynamicSmemBytes = oasis::kVerSmem;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = oasis::kVerMaxCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    // How many clusters of 16 the device holds at once: more than 8 CTAs are not promised (0 where a partition's SMs are
    // too few), and those that do not fit would run one after another.
    static OncePerDevice once;
    static int wide_on[64];
    int wide = 0;
    if (int rc = once([&] {
            if (int rc = set_smem(oasis::verify_tree_kernel, oasis::kVerSmem, "verify_tree smem")) return rc;
            const cudaError_t e =
                cudaFuncSetAttribute(oasis::verify_tree_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return cuda_fail(e, "verify_tree cluster size");
            cfg.gridDim = dim3(oasis::kVerMaxCluster);
            if (cudaOccupancyMaxActiveClusters(&wide, oasis::verify_tree_kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                wide = 0;
            }
            int dev = 0;
            if (cudaGetDevice(&dev) == cudaSuccess && dev < 64) wide_on[dev] = wide;
            return static_cast<int>(OASIS_OK);
        }))
        return rc;
    if (wide == 0) {
        int dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess && dev < 64) wide = wide_on[dev];
    }
    oasis::VerifyArgs a;
    a.probs = probs;
    a.draft = draft_probs;
    a.tokens = tokens;
    a.parent = parent;
    a.n_nodes = n_nodes;
    a.u_accept = u_accept;
    a.u_sample = u_sample;
    a.path = path;
    a.n_accept = n_accept;
    a.next_token = next_token;
    a.row_stride = static_cast<long long>(row_stride);
    a.B = d.B;
    a.T = n_tree;
    a.vocab = vocab;
    // 16 CTAs a sequence where the rows are long and all sequences' CTAs find an SM of their own, else 8 (two CTAs
    // fit an SM: 32 sequences' clusters of 8 run at once).  Trees of 8, us with 16 / 8: 151,669 entries and draft rows,
    // 1 sequence 12.7 / 15.4, 9 sequences 22.5 / 24.3, 16 sequences 26.0 / 24.5; without draft rows 11.2 / 13.3,
    // 14.5 / 15.1, 21.1 / 17.1; 32,000 entries, 1 sequence 10.1 / 10.1, 9 sequences 13.0 / 12.8.
    const int cluster = vocab > 65536 && 16ll * d.B <= sm_count() && d.B <= wide ? 16 : 8;
    cfg.gridDim = dim3(static_cast<unsigned>(d.B) * cluster);
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr.val.clusterDim.x = cluster;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, oasis::verify_tree_kernel, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail(e, "verify_tree launch");
    }
    return check_launch("verify_tree launch");
}

int oasis_commit_path(const oasis_dims* dp, int32_t n_tree, const oasis_layer* layers, int32_t n_layers,
                      const void* k_tree, const void* v_tree, const int32_t* path, const int32_t* n_accept,
                      const int32_t* ctx_len, int32_t* ctx_len_out, void* stream) {
    Dims d;
    if (int rc = check_tree(dp, n_tree, &d)) return rc;
    if (layers == nullptr) return fail(OASIS_EINVAL, "layers is NULL");
    if (n_layers < 1) return fail(OASIS_EINVAL, "n_layers must be >= 1 (got %d)", n_layers);
    if (int rc = check_ptr(k_tree, "k_tree")) return rc;
    if (int rc = check_ptr(v_tree, "v_tree")) return rc;
    if (int rc = check_ptr(path, "path")) return rc;
    if (int rc = check_ptr(n_accept, "n_accept")) return rc;
    if (int rc = check_ptr(ctx_len, "ctx_len")) return rc;
    if (int rc = check_ptr(ctx_len_out, "ctx_len_out", true)) return rc;
    if (ctx_len_out != nullptr && ctx_len_out == ctx_len)
        return fail(OASIS_EINVAL, "ctx_len_out must not alias ctx_len");
    // Every layer is checked before the first launch; the addresses of up to 64 are kept from that.
    oasis::CommitLayers c = {};
    auto take = [&](int i, int to) {
        const oasis_layer& L = layers[i];
        if (int rc = check_ptr(L.host_kv, "host_kv", true)) return rc;
        if (int rc = check_ptr(L.kmin, "kmin")) return rc;
        if (int rc = check_ptr(L.kmax, "kmax")) return rc;
        if (int rc = check_ptr(L.pool, "pool", true)) return rc;
        if (L.pool != nullptr && L.slot_table == nullptr) return fail(OASIS_EINVAL, "slot_table is NULL");
        // (read an entry at a time: a layer's slice of a stacked table starts anywhere)
        if (L.pool != nullptr && reinterpret_cast<uintptr_t>(L.slot_table) % 4 != 0)
            return fail(OASIS_EINVAL, "slot_table is not 4-byte aligned");
        const void* hv = nullptr;
        if (L.host_kv != nullptr)
            if (int rc = device_view(L.host_kv, "host_kv", false, &hv)) return rc;
        c.host[to] = static_cast<uint4*>(const_cast<void*>(hv));
        c.pool[to] = static_cast<uint4*>(L.pool);
        c.kmin[to] = static_cast<uint4*>(const_cast<void*>(L.kmin));
        c.kmax[to] = static_cast<uint4*>(const_cast<void*>(L.kmax));
        c.slot_table[to] = L.slot_table;
        return static_cast<int>(OASIS_OK);
    };
    for (int i = 0; i < n_layers; ++i)
        if (int rc = take(i, i % oasis::kCommitLayers)) return rc;
    static OncePerDevice once;
    if (int rc = once([] { return carveout(oasis::commit_path_kernel, "commit_path carve-out"); })) return rc;
    const size_t layer_rows = static_cast<size_t>(d.B) * d.Hkv * n_tree;
    for (int l0 = 0; l0 < n_layers; l0 += oasis::kCommitLayers) {
        const int nl = std::min(n_layers - l0, oasis::kCommitLayers);
        for (int i = 0; i < nl && n_layers > oasis::kCommitLayers; ++i)
            if (int rc = take(l0 + i, i)) return rc;
        const dim3 grid(static_cast<unsigned>(d.B * d.Hkv), static_cast<unsigned>(nl));
        oasis::commit_path_kernel<<<grid, oasis::kCommitThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            c, d, n_tree, static_cast<const uint4*>(k_tree) + l0 * layer_rows * 16,
            static_cast<const uint4*>(v_tree) + l0 * layer_rows * 16, path, n_accept, ctx_len,
            l0 == 0 ? ctx_len_out : nullptr);
        if (int rc = check_launch("commit_path launch")) return rc;
    }
    return OASIS_OK;
}

}  // extern "C"
