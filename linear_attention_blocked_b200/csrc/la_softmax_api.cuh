// la_softmax_api.cuh -- C entry points of the softmax-attention operators and
// the paged key/value cache: argument checks, workspaces, tensor maps and
// launches.  Part of la_lib.cu (uses its helpers and status word).
#pragma once

namespace {

SmemAttr g_attr_softmax, g_attr_softmax_dkv, g_attr_softmax_dq;

struct SoftmaxLayout {
    size_t hdr, prefix, entries, total;
    long long emax;
};

// Tables of the scheduler: at most one ragged block per sequence.  Sized for
// 128-row entries, which also covers entries of 256 rows.
SoftmaxLayout softmax_layout(int nseq, long long T) {
    SoftmaxLayout w;
    w.emax = T / la::BLK + nseq;
    w.hdr = 0;
    w.prefix = la::HDR_BYTES;
    w.entries = w.prefix + round_up(((size_t)nseq + 1) * sizeof(int), 256);
    w.total = w.entries + round_up((size_t)w.emax * sizeof(int4), 256);
    return w;
}

// Work items of the prompt kernel: pairs of query tiles.  With no more items
// than SMs every CTA has one, which it finds itself: no scheduler launch
// and no workspace (129 tokens, 64 heads over 8: 14.4 us with, 12.3 us without; back
// to back, with the next call set up meanwhile, 10.2 us).  The count is a bound, half
// an entry per sequence too high on average: where the likely count fits and items
// are short, those too many wait for an SM (9 sequences of up to 500, 8 heads over 8,
// at most 152 items: 19.2 us with the scheduler, 15.9 us without; a second wave
// that really comes costs more: 700 tokens, 64 heads over 8, 192 items, 22.2 / 25.2).
// Depends on the shape only, so that the workspace size does.
struct SoftmaxItems {
    int rows, pairs;   // rows per entry, pairs per entry and key/value head
    long long items;
    bool direct;
    bool split;
};

// With few items of many key tiles the tiles are cut into equal runs, one per SM,
// and cut items joined by a second kernel.  Whole items / runs, us: 16 new tokens,
// 64 heads over 8, behind 2000 35 / 23, behind 16000 215 / 63; 128 behind 60000 787 /
// 243; 256 behind 8000 118 / 83; a prompt of 8000, 2 heads 111 / 57.  From 100 items on
// the runs are hardly shorter than the items (500 behind 8000, 128 items: 123 / 161),
// and below 14 tiles the second launch costs what they save (prompt of 1600, 8 heads
// over 1: 29 / 32).
constexpr size_t kSplitParts = (size_t)la::SMX_CTAS * 2 * 2 * la::BLK * la::SMX_PART * sizeof(float);
constexpr size_t kSplitWs = kSplitParts + (size_t)la::SMX_CTAS * 3 * sizeof(int4);

// keys: a bound on the keys of a row
SoftmaxItems softmax_items(int nseq, long long T, long long keys, int H, int Hkv) {
    const int G = H / Hkv;
    SoftmaxItems s;
    s.rows = G % 2 ? 2 * la::BLK : la::BLK;
    s.pairs = G % 2 ? G : G / 2;
    const long long per = (long long)Hkv * s.pairs;
    s.items = (T + (long long)nseq * (s.rows - 1)) / s.rows * per;
    s.direct = T > 0 && (s.items <= 148 || (keys <= 1024 && s.items - (nseq - 1) * per / 2 <= 148));
    s.split = s.direct && s.items <= 96 && keys > 13 * la::BLK;
    return s;
}

// Order of the work items of packed sequences.  By length, the longest of all
// heads and sequences first, leaves the SMs the least to wait for at the end;
// key/value head by head and sequence by sequence lets the CTAs at work share keys
// and values in L2, which matters where they do not all fit there (126 MB).  By
// length / by head, forward: 3 sequences of up to 3000, 16 heads over 16, 58 / 75 us; 4
// of up to 600, 64 over 8, 27 / 32 us; 12 of up to 1500, 64 over 8, 230 / 235 us.  The
// backward pass, whose two kernels fill each other's ends, gains only where its
// key blocks are few (those cases: 160 / 165, 88 / 90, but 866 / 830 us).
bool softmax_by_length(int nseq, long long T, int Hkv) {
    return T * Hkv <= 131072 && nseq <= la::SCHED_THREADS && T <= (long long)la::SCHED_THREADS * la::BLK;
}

la_status check_softmax(int H, int Hkv, int d, float scale) {
    if (H <= 0 || Hkv <= 0 || d <= 0 || H % Hkv) return LA_ERR_INVALID_ARGUMENT;
    if (!(scale > 0.f) || scale > 1.0e38f) return LA_ERR_INVALID_ARGUMENT;  // also rejects NaN
    if (d != la::D) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

constexpr float kLog2e = 1.44269504088896341f;

int *status_word() {
    static std::atomic<int *> cached[kMaxDevices];  // the address is fixed per device
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return nullptr;
    if (dev < kMaxDevices && cached[dev].load()) return cached[dev].load();
    int *status = nullptr;
    if (cudaGetSymbolAddress(reinterpret_cast<void **>(&status), g_la_status) != cudaSuccess) return nullptr;
    if (dev < kMaxDevices) cached[dev].store(status);
    return status;
}

// A paged cache [n_pages, Hkv, page, 128] viewed as {64 features, rows, 2
// halves}: a box {64, rows, 1} is one half of `box_rows` keys of one page.
bool encode_page_map(CUtensorMap *map, const void *base, long long rows, int box_rows) {
    EncodeTiledFn fn = get_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, 2};
    const cuuint64_t strides[2] = {(cuuint64_t)la::D * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A paged cache as the entry points take it.
struct PagedCache {
    void *k, *v;
    int n_pages, page;
    const int *table;
    int max_pages;
    const int *lens;
};

size_t cache_bytes(const PagedCache &c, int Hkv) { return (size_t)c.n_pages * Hkv * c.page * la::D * 2; }

bool page_size_built(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

la_status check_cache(const PagedCache &c, int Hkv) {
    if (c.n_pages <= 0 || c.max_pages <= 0 || c.page <= 0) return LA_ERR_INVALID_ARGUMENT;
    if (!page_size_built(c.page)) return LA_ERR_UNSUPPORTED;
    if (!c.k || !c.v || !c.table || !c.lens) return LA_ERR_INVALID_ARGUMENT;
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.table, 4) || !aligned(c.lens, 4))
        return LA_ERR_INVALID_ARGUMENT;
    // rows of the cache are tensor-map coordinates
    if ((long long)c.n_pages * Hkv * c.page > 0x7fffffffLL || (long long)c.max_pages * c.page > 0x7fffffffLL)
        return LA_ERR_UNSUPPORTED;
    const size_t n = cache_bytes(c, Hkv);
    return ranges_overlap(c.k, n, c.v, n) ? LA_ERR_INVALID_ARGUMENT : LA_OK;
}

// Is the written range [w, w + n) clear of q, k, v and (with one) the cache?
struct SoftmaxInputs {
    const void *q, *k, *v;
    size_t n_q, n_kv;
    const PagedCache *cache;
    size_t n_cache;
};

bool clear_of(const void *w, size_t n, const SoftmaxInputs &in) {
    if (ranges_overlap(w, n, in.q, in.n_q) || ranges_overlap(w, n, in.k, in.n_kv) || ranges_overlap(w, n, in.v, in.n_kv))
        return false;
    return !in.cache || (!ranges_overlap(w, n, in.cache->k, in.n_cache) && !ranges_overlap(w, n, in.cache->v, in.n_cache));
}

// Launch a kernel that may be set up while the one before it in the stream
// still runs (it waits for that one's end itself, with griddepcontrol.wait).
template <class... P, class... A>
bool launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// Shared body of la_softmax_prefill_varlen and, with a cache, la_softmax_prefill_paged.
la_status softmax_prefill_impl(const void *q, const void *k, const void *v, const int *cu, int nseq, long long T,
                               int max_seqlen, int H, int Hkv, int d, float scale, const PagedCache *cache, void *out,
                               float *lse, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    la_status st = check_softmax(H, Hkv, d, scale);
    if (st != LA_OK) return st;
    if (nseq < 0 || T < 0 || max_seqlen < 0) return LA_ERR_INVALID_ARGUMENT;
    if (nseq == 0) return T == 0 ? LA_OK : LA_ERR_INVALID_ARGUMENT;
    if (!cu || !aligned(cu, 4)) return LA_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!q || !k || !v || !out)) return LA_ERR_INVALID_ARGUMENT;
    const void *ptrs[4] = {q, k, v, out};
    for (const void *p : ptrs)
        if (p && !aligned(p, 16)) return LA_ERR_INVALID_ARGUMENT;
    if (lse && !aligned(lse, 4)) return LA_ERR_INVALID_ARGUMENT;
    if (cache && (st = check_cache(*cache, Hkv)) != LA_OK) return st;
    const size_t n_q = (size_t)T * H * la::D * 2, n_kv = (size_t)T * Hkv * la::D * 2, n_lse = (size_t)T * H * 4;
    const SoftmaxInputs in = {q, k, v, n_q, n_kv, cache, cache ? cache_bytes(*cache, Hkv) : 0};
    if (!clear_of(out, n_q, in) || !clear_of(lse, n_lse, in) || ranges_overlap(lse, n_lse, out, n_q))
        return LA_ERR_INVALID_ARGUMENT;
    if (cache && (ranges_overlap(cache->k, in.n_cache, q, n_q) || ranges_overlap(cache->k, in.n_cache, k, n_kv) ||
                  ranges_overlap(cache->k, in.n_cache, v, n_kv) || ranges_overlap(cache->v, in.n_cache, q, n_q) ||
                  ranges_overlap(cache->v, in.n_cache, k, n_kv) || ranges_overlap(cache->v, in.n_cache, v, n_kv)))
        return LA_ERR_INVALID_ARGUMENT;
    const long long max_keys = cache ? (long long)cache->max_pages * cache->page : 0;
    const SoftmaxItems it = softmax_items(nseq, T, cache ? max_keys : (max_seqlen < T ? max_seqlen : T), H, Hkv);
    const SoftmaxLayout w = softmax_layout(nseq, T);
    const size_t need = it.split ? kSplitWs : it.direct ? 0 : w.total;
    if (need) {
        if (!workspace || ws_bytes < need) return LA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return LA_ERR_INVALID_ARGUMENT;
        if (!clear_of(workspace, need, in) || ranges_overlap(workspace, need, out, n_q) ||
            ranges_overlap(workspace, need, lse, n_lse))
            return LA_ERR_INVALID_ARGUMENT;
    }
    const int G = H / Hkv, rows = it.rows, pairs = it.pairs;
    const bool direct = it.direct;
    const long long items = it.items;
    if (items > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    int *status = status_word();
    if (!status) return LA_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);

    const int sms = device_sm_count();
    la::SoftmaxScheduleParams sp;
    sp.cu = cu;
    sp.past = cache ? cache->lens : nullptr;
    sp.nseq = nseq;
    sp.T = (int)T;
    sp.max_seqlen = max_seqlen;
    sp.max_keys = max_keys;
    sp.rows = rows;
    sp.items_per_entry = Hkv * pairs;
    sp.by_length = !cache && softmax_by_length(nseq, T, Hkv);
    sp.hdr = reinterpret_cast<int *>(ws + w.hdr);
    sp.prefix = reinterpret_cast<int *>(ws + w.prefix);
    sp.entries = reinterpret_cast<int4 *>(ws + w.entries);
    sp.status = status;
    if (!direct) {  // (without tokens only the tables are checked)
        if (!launch_dependent(la::la_softmax_schedule_kernel, dim3(1), la::SCHED_THREADS, 0, stream, sp)) return LA_ERR_CUDA;
        ++g_launches;
        if (T == 0) return LA_OK;
    }

    CUtensorMap mq, mk, mv, mkc, mvc;
    if (!encode_qkv_map(&mq, q, (int)T, H) || !encode_qkv_map(&mk, k, (int)T, Hkv) ||
        !encode_qkv_map(&mv, v, (int)T, Hkv))
        return LA_ERR_CUDA;
    la::SoftmaxPrefillParams pp;
    memset(&pp, 0, sizeof pp);
    if (cache) {
        const long long cache_rows = (long long)cache->n_pages * Hkv * cache->page;
        if (!encode_page_map(&mkc, cache->k, cache_rows, cache->page) ||
            !encode_page_map(&mvc, cache->v, cache_rows, cache->page))
            return LA_ERR_CUDA;
        pp.past = cache->lens;
        pp.pages = cache->table;
        pp.max_pages = cache->max_pages;
        pp.n_pages = cache->n_pages;
        pp.page = cache->page;
        pp.page_shift = log2_of(cache->page);
        pp.kc = static_cast<__nv_bfloat16 *>(cache->k);
        pp.vc = static_cast<__nv_bfloat16 *>(cache->v);
        if (direct) {
            pp.new_k = static_cast<const __nv_bfloat16 *>(k);
            pp.new_v = static_cast<const __nv_bfloat16 *>(v);
        } else {
            const la::AppendTables at = {static_cast<const __nv_bfloat16 *>(k), static_cast<const __nv_bfloat16 *>(v),
                                         pp.kc, pp.vc, cu, cache->table, cache->lens, nseq, Hkv, cache->max_pages,
                                         cache->n_pages, cache->page, pp.page_shift, status};
            const long long blocks = (T * Hkv * (la::D / 8) + la::APPEND_THREADS - 1) / la::APPEND_THREADS;
            if (!launch_dependent(la::la_cache_append_kernel, dim3((unsigned)(blocks < 148 * 8 ? blocks : 148 * 8)),
                                  la::APPEND_THREADS, 0, stream, at, (int)T, static_cast<const int *>(sp.hdr)))
                return LA_ERR_CUDA;
            ++g_launches;
        }
    } else {
        mkc = mk;
        mvc = mv;
    }
    pp.out = static_cast<__nv_bfloat16 *>(out);
    pp.lse = lse;
    pp.hdr = sp.hdr;
    pp.entries = sp.entries;
    pp.H = H;
    pp.Hkv = Hkv;
    pp.G = G;
    pp.pairs = pairs;
    pp.rows = rows;
    pp.by_length = sp.by_length;
    pp.scale_log2 = scale * kLog2e;
    pp.wait_limit_ns = g_wait_limit_ns.load();
    pp.status = status;
    pp.direct = direct;
    pp.split = it.split;
    if (it.split) {
        pp.parts = reinterpret_cast<float *>(ws);
        pp.info = reinterpret_cast<int4 *>(ws + kSplitParts);
    }
    pp.cu = cu;
    pp.nseq = nseq;
    pp.T = (int)T;
    pp.max_seqlen = max_seqlen;
    pp.max_keys = max_keys;
    st = ensure_smem_attr(g_attr_softmax, la::la_softmax_prefill_kernel, la::SMX_SMEM);
    if (st != LA_OK) return st;
    const long long grid = it.split ? la::SMX_CTAS : direct ? items : sms;
    if (!launch_dependent(la::la_softmax_prefill_kernel, dim3((unsigned)grid), la::SMX_THREADS, la::SMX_SMEM, stream, mq,
                          mk, mv, mkc, mvc, pp))
        return LA_ERR_CUDA;
    ++g_launches;
    if (it.split) {
        const int tile_rows = max_seqlen < la::BLK ? max_seqlen : la::BLK;
        const unsigned z = (unsigned)(tile_rows + la::SPLIT_JOIN_ROWS - 1) / la::SPLIT_JOIN_ROWS;
        if (!launch_dependent(la::la_softmax_split_join_kernel, dim3(la::SMX_CTAS, 2, z ? z : 1),
                              32 * la::SPLIT_JOIN_ROWS, 0, stream, pp))
            return LA_ERR_CUDA;
        ++g_launches;
    }
    return LA_OK;
}

constexpr size_t kDecodeParts = (size_t)la::SD_CTAS * 2 * la::SD_PART * sizeof(float);
constexpr size_t kDecodeWs = kDecodeParts + (size_t)la::SD_CTAS * sizeof(int4);

int decode_heads(int G) { return G > la::SD_NARROW ? la::SD_WIDE : la::SD_NARROW; }

// CTAs (a cluster) that a row of a decode step takes, 0 for the form that cuts
// all rows' tiles into equal runs and joins them with a second kernel.  CTAs per
// row need no second kernel and leave their order to the hardware's scheduler,
// but a row that is much longer than the others holds them up, and few rows do
// not fill the GPU: so the largest cluster that keeps all CTAs resident, and rows
// of at most some 2048 keys per CTA.  64 heads over 8, us, rows of the length given
// (in brackets: of lengths up to it), in that form / in runs: 1 request of 64 keys
// 5.7 / 8.3, of 4000 9.8 / 18.5, of 32000 (cluster of 16) 27.6 / 37.4; 4 of 16000 43
// [29] / 49 [33]; 9 of 2000 15.4 [13.8] / 18.0 [13.9], of 8000 48 [38] / 53 [31]; 18 of
// 1000 13.4 [11.8] / 18.7 [13.9], of 4000 47 [34] / 53 [30]; 32 of 4000 81 [48] / 87 [48];
// 256 of 4000 582 [293] / 615 [316], of 8000 no difference.  Clusters of 16 only while
// one wave of them fits (2 requests of 700 keys: 13.8 against 7.7 in clusters of 8)
// and for rows whose reading outweighs their longer meeting (1 request of 16000 keys
// 17.5 against 20.0 in a cluster of 8, of 64 keys 7.3 against 5.7).
int decode_cluster(long long B, int H, int Hkv, long long max_keys) {
    const int G = H / Hkv, heads = decode_heads(G), chunks = (G + heads - 1) / heads;
    const long long rows = B * Hkv * chunks;
    if (rows * 16 <= 148 && max_keys > 4096) return max_keys <= 32768 ? 16 : 0;
    for (int c = 8; c > 1; c /= 2)
        if (rows * c <= 256) return max_keys <= 2048 * c ? c : 0;
    return max_keys <= (rows >= 256 ? 4096 : 2048) ? 1 : 0;
}

template <int HEADS, int STAGES, int CLUSTER>
la_status launch_decode_cluster(const CUtensorMap &mk, const CUtensorMap &mv, const la::SoftmaxDecodeParams &dp,
                                cudaStream_t stream) {
    using S = la::DecodeShape<HEADS, STAGES>;
    static SmemAttr attr;
    auto kernel = la::la_softmax_decode_cluster_kernel<HEADS, STAGES, CLUSTER>;
    la_status st = ensure_smem_attr(attr, kernel, S::SMEM, CLUSTER > 8);
    if (st != LA_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)dp.B * dp.Hkv * dp.chunks * CLUSTER));
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2] = {};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = CLUSTER;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = CLUSTER > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, mk, mv, dp) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

template <int HEADS, int STAGES>
la_status launch_decode_rows(int cluster, const CUtensorMap &mk, const CUtensorMap &mv,
                             const la::SoftmaxDecodeParams &dp, cudaStream_t stream) {
    switch (cluster) {
    case 8: return launch_decode_cluster<HEADS, STAGES, 8>(mk, mv, dp, stream);
    case 4: return launch_decode_cluster<HEADS, STAGES, 4>(mk, mv, dp, stream);
    case 2: return launch_decode_cluster<HEADS, STAGES, 2>(mk, mv, dp, stream);
    default: return launch_decode_cluster<HEADS, STAGES, 1>(mk, mv, dp, stream);
    }
}

template <int HEADS>
la_status launch_decode(int cluster, const CUtensorMap &mk, const CUtensorMap &mv, const la::SoftmaxDecodeParams &dp,
                        cudaStream_t stream) {
    if (cluster == 16) return launch_decode_cluster<HEADS, 3, 16>(mk, mv, dp, stream);
    if (cluster) {
        // The deep ring where CTAs have an SM each (clusters of them need room in one
        // part of the GPU, so fewer) and more tiles than the short ring holds.  64 heads
        // over 8, deep / short: 1 request of 4000 keys, one CTA a row, 31.5 / 36 us; of 16000,
        // clusters of 8, 20.0 / 23; 2 of 3000 in clusters of 8 12.7 / 8.8; 1 of 700 7.2 / 6.3.
        const long long ctas = (long long)dp.B * dp.Hkv * dp.chunks * cluster;
        const bool deep = ctas <= (cluster == 1 ? 148 : 96) && dp.max_keys > 3 * la::SD_KEYS * cluster;
        return deep ? launch_decode_rows<HEADS, 6>(cluster, mk, mv, dp, stream)
                    : launch_decode_rows<HEADS, 3>(cluster, mk, mv, dp, stream);
    }
    using S = la::DecodeShape<HEADS, 3>;
    static SmemAttr attr;
    auto kernel = la::la_softmax_decode_kernel<HEADS>;
    la_status st = ensure_smem_attr(attr, kernel, S::SMEM);
    if (st != LA_OK) return st;
    return launch_dependent(kernel, dim3(la::SD_CTAS), S::THREADS, S::SMEM, stream, mk, mv, dp) ? LA_OK : LA_ERR_CUDA;
}

}  // namespace

namespace {

// Workspace of the prompt kernel for rows of up to `keys` keys: of a call that
// knows a smaller bound at most this.
size_t softmax_ws(int nseq, long long T, long long keys, int H, int Hkv) {
    const SoftmaxItems it = softmax_items(nseq, T, keys, H, Hkv);
    return it.split ? kSplitWs : it.direct ? 0 : softmax_layout(nseq, T).total;
}

}  // namespace

size_t la_softmax_prefill_varlen_workspace_size(int nseq, int total_tokens, int H, int Hkv, int d) {
    if (nseq < 0 || total_tokens < 0 || check_softmax(H, Hkv, d, 1.f) != LA_OK) return 0;
    return softmax_ws(nseq, total_tokens, total_tokens, H, Hkv);
}

la_status la_softmax_prefill_varlen(const void *q, const void *k, const void *v, const int *cu_seqlens, int nseq,
                                    int total_tokens, int max_seqlen, int H, int Hkv, int d, float scale, void *out,
                                    float *lse, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    return softmax_prefill_impl(q, k, v, cu_seqlens, nseq, total_tokens, max_seqlen, H, Hkv, d, scale, nullptr, out,
                                lse, workspace, ws_bytes, stream);
}

size_t la_softmax_prefill_paged_workspace_size(int nseq, int total_tokens, int H, int Hkv, int d, int page_size,
                                               int max_pages) {
    if (nseq < 0 || total_tokens < 0 || check_softmax(H, Hkv, d, 1.f) != LA_OK || page_size <= 0 || max_pages <= 0)
        return 0;
    return softmax_ws(nseq, total_tokens, (long long)page_size * max_pages, H, Hkv);
}

la_status la_softmax_prefill_paged(const void *q, const void *k, const void *v, const int *cu_seqlens, int nseq,
                                   int total_tokens, int max_seqlen, int H, int Hkv, int d, float scale,
                                   void *k_cache, void *v_cache, int n_pages, int page_size, const int *page_table,
                                   int max_pages, const int *cache_lens, void *out, float *lse, void *workspace,
                                   size_t ws_bytes, cudaStream_t stream) {
    const PagedCache cache = {k_cache, v_cache, n_pages, page_size, page_table, max_pages, cache_lens};
    return softmax_prefill_impl(q, k, v, cu_seqlens, nseq, total_tokens, max_seqlen, H, Hkv, d, scale, &cache, out,
                                lse, workspace, ws_bytes, stream);
}

size_t la_softmax_decode_paged_workspace_size(int B, int H, int Hkv, int d, int page_size, int max_pages) {
    if (B <= 0 || check_softmax(H, Hkv, d, 1.f) != LA_OK || page_size <= 0 || max_pages <= 0) return 0;
    return decode_cluster(B, H, Hkv, (long long)page_size * max_pages) ? 0 : kDecodeWs;
}

la_status la_softmax_decode_paged(const void *q, const void *k, const void *v, int B, int H, int Hkv, int d,
                                  float scale, void *k_cache, void *v_cache, int n_pages, int page_size,
                                  const int *page_table, int max_pages, const int *cache_lens, void *out,
                                  la_dtype out_dtype, float *lse, void *workspace, size_t ws_bytes,
                                  cudaStream_t stream) {
    la_status st = check_softmax(H, Hkv, d, scale);
    if (st != LA_OK) return st;
    if (B < 0 || (out_dtype != LA_BF16 && out_dtype != LA_FP32)) return LA_ERR_INVALID_ARGUMENT;
    if (B == 0) return LA_OK;
    if (!q || !k || !v || !out) return LA_ERR_INVALID_ARGUMENT;
    const void *ptrs[4] = {q, k, v, out};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return LA_ERR_INVALID_ARGUMENT;
    if (lse && !aligned(lse, 4)) return LA_ERR_INVALID_ARGUMENT;
    const PagedCache cache = {k_cache, v_cache, n_pages, page_size, page_table, max_pages, cache_lens};
    if ((st = check_cache(cache, Hkv)) != LA_OK) return st;
    const size_t esz = out_dtype == LA_FP32 ? 4 : 2;
    const size_t n_q = (size_t)B * H * la::D * 2, n_kv = (size_t)B * Hkv * la::D * 2, n_lse = (size_t)B * H * 4;
    const size_t n_out = (size_t)B * H * la::D * esz;
    const SoftmaxInputs in = {q, k, v, n_q, n_kv, &cache, cache_bytes(cache, Hkv)};
    if (!clear_of(out, n_out, in) || !clear_of(lse, n_lse, in) || ranges_overlap(lse, n_lse, out, n_out) ||
        !clear_of(cache.k, in.n_cache, {q, k, v, n_q, n_kv, nullptr, 0}) ||
        !clear_of(cache.v, in.n_cache, {q, k, v, n_q, n_kv, nullptr, 0}))
        return LA_ERR_INVALID_ARGUMENT;
    const int cluster = decode_cluster(B, H, Hkv, (long long)max_pages * page_size);
    if (!cluster) {
        if (!workspace || ws_bytes < kDecodeWs) return LA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return LA_ERR_INVALID_ARGUMENT;
        if (!clear_of(workspace, kDecodeWs, in) || ranges_overlap(workspace, kDecodeWs, out, n_out) ||
            ranges_overlap(workspace, kDecodeWs, lse, n_lse))
            return LA_ERR_INVALID_ARGUMENT;
    }
    int *status = status_word();
    if (!status) return LA_ERR_CUDA;
    const long long cache_rows = (long long)n_pages * Hkv * page_size;
    const int box = page_size < la::SD_KEYS ? page_size : la::SD_KEYS;
    CUtensorMap mk, mv;
    if (!encode_page_map(&mk, k_cache, cache_rows, box) || !encode_page_map(&mv, v_cache, cache_rows, box))
        return LA_ERR_CUDA;
    la::SoftmaxDecodeParams dp;
    dp.q = static_cast<const __nv_bfloat16 *>(q);
    dp.k = static_cast<const __nv_bfloat16 *>(k);
    dp.v = static_cast<const __nv_bfloat16 *>(v);
    dp.kc = static_cast<__nv_bfloat16 *>(k_cache);
    dp.vc = static_cast<__nv_bfloat16 *>(v_cache);
    dp.pages = page_table;
    dp.lens = cache_lens;
    dp.out = out;
    dp.lse = lse;
    dp.parts = static_cast<float *>(workspace);
    dp.info = reinterpret_cast<int4 *>(static_cast<uint8_t *>(workspace) + kDecodeParts);
    dp.out_fp32 = out_dtype == LA_FP32;
    dp.B = B;
    dp.H = H;
    dp.Hkv = Hkv;
    dp.G = H / Hkv;
    dp.chunks = (dp.G + decode_heads(dp.G) - 1) / decode_heads(dp.G);
    dp.max_pages = max_pages;
    dp.n_pages = n_pages;
    dp.page = page_size;
    dp.page_shift = log2_of(page_size);
    dp.max_keys = (long long)max_pages * page_size;
    dp.scale_log2 = scale * kLog2e;
    dp.wait_limit_ns = g_wait_limit_ns.load();
    dp.status = status;
    st = decode_heads(dp.G) == la::SD_WIDE ? launch_decode<la::SD_WIDE>(cluster, mk, mv, dp, stream)
                                           : launch_decode<la::SD_NARROW>(cluster, mk, mv, dp, stream);
    if (st != LA_OK) return st;
    ++g_launches;
    if (cluster) return LA_OK;
    if (!launch_dependent(la::la_softmax_join_kernel, dim3(la::SD_CTAS, dp.G < la::SD_WIDE ? dp.G : la::SD_WIDE),
                          la::D, 0, stream, dp))
        return LA_ERR_CUDA;
    ++g_launches;
    return LA_OK;
}

la_status la_cache_copy_pages(void *k_cache, void *v_cache, int n_pages, int page_size, int Hkv, int d,
                              const int *src, const int *dst, int n, cudaStream_t stream) {
    if (n_pages <= 0 || page_size <= 0 || Hkv <= 0 || d <= 0 || n < 0) return LA_ERR_INVALID_ARGUMENT;
    if (d != la::D || !page_size_built(page_size)) return LA_ERR_UNSUPPORTED;
    if (n == 0) return LA_OK;
    if (!k_cache || !v_cache || !src || !dst || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(src, 4) ||
        !aligned(dst, 4))
        return LA_ERR_INVALID_ARGUMENT;
    const size_t page_bytes = (size_t)Hkv * page_size * la::D * 2, bytes = page_bytes * n_pages;
    if (ranges_overlap(k_cache, bytes, v_cache, bytes)) return LA_ERR_INVALID_ARGUMENT;
    int *status = status_word();
    if (!status) return LA_ERR_CUDA;
    const long long pieces = (long long)((page_bytes + la::COPY_PIECE - 1) / la::COPY_PIECE);
    const long long blocks = 2 * pieces * n, most = 148 * 16;
    if (!launch_dependent(la::la_cache_copy_kernel, dim3((unsigned)(blocks < most ? blocks : most)), la::COPY_THREADS, 0,
                          stream, static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), src, dst, n, n_pages,
                          (long long)page_bytes, status))
        return LA_ERR_CUDA;
    ++g_launches;
    return LA_OK;
}

namespace {

// Workspace of the backward pass: the scheduler's tables, lse2 and delta, and
// the fp32 sums of dk and dv where several CTAs share a key block.
struct SoftmaxBwdLayout {
    SoftmaxLayout tables;
    size_t lse2, delta, parts, total;
    int nparts;
};

SoftmaxBwdLayout softmax_bwd_layout(int nseq, long long T, int H, int Hkv) {
    SoftmaxBwdLayout w;
    w.tables = softmax_layout(nseq, T);
    const size_t rows = round_up((size_t)T * H * sizeof(float), 256);
    w.lse2 = w.tables.total;
    w.delta = w.lse2 + rows;
    w.parts = w.delta + rows;
    const int G = H / Hkv;
    // The longest walk of dk and dv, over all of a sequence's rows for all of a
    // group's heads, should be short against an SM's share of the whole: with one
    // sequence it is 169 / items of that share.  (With many items one part is
    // faster, 2.32 against 2.38 ms with two at 16908 tokens of 32 heads over 4:
    // dq fills the SMs that run out, and no sums go through memory.)
    const long long items = w.tables.emax * Hkv;
    w.nparts = 1;
    while (2 * w.nparts <= G && items * w.nparts < 2 * 148) w.nparts *= 2;
    w.total = w.parts + (w.nparts > 1 ? (size_t)w.nparts * 2 * T * Hkv * la::D * sizeof(float) : 0);
    return w;
}

}  // namespace

size_t la_softmax_prefill_backward_varlen_workspace_size(int nseq, int total_tokens, int H, int Hkv, int d) {
    if (nseq < 0 || total_tokens < 0 || check_softmax(H, Hkv, d, 1.f) != LA_OK) return 0;
    return softmax_bwd_layout(nseq, total_tokens, H, Hkv).total;
}

la_status la_softmax_prefill_backward_varlen(const void *q, const void *k, const void *v, const void *out,
                                             const float *lse, const void *dout, const int *cu_seqlens, int nseq,
                                             int total_tokens, int max_seqlen, int H, int Hkv, int d, float scale,
                                             void *dq, void *dk, void *dv, void *workspace, size_t ws_bytes,
                                             cudaStream_t stream) {
    la_status st = check_softmax(H, Hkv, d, scale);
    if (st != LA_OK) return st;
    const long long T = total_tokens;
    if (nseq < 0 || T < 0 || max_seqlen < 0) return LA_ERR_INVALID_ARGUMENT;
    if (nseq == 0) return T == 0 ? LA_OK : LA_ERR_INVALID_ARGUMENT;
    if (!cu_seqlens || !aligned(cu_seqlens, 4)) return LA_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv)) return LA_ERR_INVALID_ARGUMENT;
    const void *ptrs[8] = {q, k, v, out, dout, dq, dk, dv};
    for (const void *p : ptrs)
        if (p && !aligned(p, 16)) return LA_ERR_INVALID_ARGUMENT;
    if (lse && !aligned(lse, 4)) return LA_ERR_INVALID_ARGUMENT;
    const size_t n_q = (size_t)T * H * la::D * 2, n_kv = (size_t)T * Hkv * la::D * 2, n_lse = (size_t)T * H * 4;
    const SoftmaxBwdLayout w = softmax_bwd_layout(nseq, T, H, Hkv);
    struct Range {
        const void *p;
        size_t n;
    };
    const Range ins[6] = {{q, n_q}, {k, n_kv}, {v, n_kv}, {out, n_q}, {lse, n_lse}, {dout, n_q}};
    const Range outs[4] = {{dq, n_q}, {dk, n_kv}, {dv, n_kv}, {workspace, w.total}};
    for (int i = 0; i < 4; ++i) {
        for (const Range &r : ins)
            if (ranges_overlap(outs[i].p, outs[i].n, r.p, r.n)) return LA_ERR_INVALID_ARGUMENT;
        for (int j = i + 1; j < 4; ++j)
            if (ranges_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return LA_ERR_INVALID_ARGUMENT;
    }
    if (!workspace || ws_bytes < w.total) return LA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return LA_ERR_INVALID_ARGUMENT;
    if (w.tables.emax * H > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    int *status = status_word();
    if (!status) return LA_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);

    la::SoftmaxScheduleParams sp;
    sp.cu = cu_seqlens;
    sp.past = nullptr;
    sp.nseq = nseq;
    sp.T = (int)T;
    sp.max_seqlen = max_seqlen;
    sp.max_keys = 0;
    sp.rows = la::BLK;
    sp.items_per_entry = 0;  // both kernels count their own
    sp.by_length = w.tables.emax * Hkv <= 2 * 148 && softmax_by_length(nseq, T, Hkv);
    sp.hdr = reinterpret_cast<int *>(ws + w.tables.hdr);
    sp.prefix = reinterpret_cast<int *>(ws + w.tables.prefix);
    sp.entries = reinterpret_cast<int4 *>(ws + w.tables.entries);
    sp.status = status;

    la::SoftmaxBwdParams bp;
    float *lse2 = reinterpret_cast<float *>(ws + w.lse2), *delta = reinterpret_cast<float *>(ws + w.delta);
    bp.lse2 = lse2;
    bp.delta = delta;
    bp.dq = static_cast<__nv_bfloat16 *>(dq);
    bp.dk = static_cast<__nv_bfloat16 *>(dk);
    bp.dv = static_cast<__nv_bfloat16 *>(dv);
    bp.parts = w.nparts > 1 ? reinterpret_cast<float *>(ws + w.parts) : nullptr;
    bp.hdr = sp.hdr;
    bp.entries = sp.entries;
    bp.T = (int)T;
    bp.H = H;
    bp.Hkv = Hkv;
    bp.G = H / Hkv;
    bp.nparts = w.nparts;
    bp.by_length = sp.by_length;
    bp.scale = scale;
    bp.scale_log2 = scale * kLog2e;
    bp.wait_limit_ns = g_wait_limit_ns.load();
    bp.status = status;

    const long long row_blocks = (T * H + la::SCHED_THREADS / 16 - 1) / (la::SCHED_THREADS / 16);
    if (!launch_dependent(la::la_softmax_rows_kernel, dim3(1 + (unsigned)(row_blocks < 148 * 4 ? row_blocks : 148 * 4)),
                          la::SCHED_THREADS, 0, stream, sp, static_cast<const __nv_bfloat16 *>(out),
                          static_cast<const __nv_bfloat16 *>(dout), lse, lse2, delta, (int)T, H))
        return LA_ERR_CUDA;
    ++g_launches;
    if (T == 0) return LA_OK;  // (the tables are checked)

    CUtensorMap mq, mk, mv, mg;
    if (!encode_qkv_map(&mq, q, (int)T, H) || !encode_qkv_map(&mk, k, (int)T, Hkv) ||
        !encode_qkv_map(&mv, v, (int)T, Hkv) || !encode_qkv_map(&mg, dout, (int)T, H))
        return LA_ERR_CUDA;
    if ((st = ensure_smem_attr(g_attr_softmax_dkv, la::la_softmax_dkv_kernel, la::DKV_SMEM)) != LA_OK) return st;
    if ((st = ensure_smem_attr(g_attr_softmax_dq, la::la_softmax_dq_kernel, la::DQ_SMEM)) != LA_OK) return st;
    const int sms = device_sm_count();
    const long long dkv_items = w.tables.emax * Hkv * (long long)w.nparts, dq_items = w.tables.emax * H;
    if (!launch_dependent(la::la_softmax_dkv_kernel, dim3((unsigned)(dkv_items < sms ? dkv_items : sms)), la::SB_THREADS,
                          la::DKV_SMEM, stream, mq, mk, mv, mg, bp))
        return LA_ERR_CUDA;
    ++g_launches;
    if (!launch_dependent(la::la_softmax_dq_kernel, dim3((unsigned)(dq_items < sms ? dq_items : sms)), la::SB_THREADS,
                          la::DQ_SMEM, stream, mq, mk, mv, mg, bp))
        return LA_ERR_CUDA;
    ++g_launches;
    if (w.nparts > 1) {
        const long long n = T * Hkv * la::D, blocks = (n / 2 + 255) / 256;
        la::la_softmax_dkv_sum_kernel<<<(unsigned)(blocks < 148 * 8 ? blocks : 148 * 8), 256, 0, stream>>>(
            bp.hdr, bp.parts, w.nparts, n, bp.dk, bp.dv);
        if (cudaGetLastError() != cudaSuccess) return LA_ERR_CUDA;
        ++g_launches;
    }
    return LA_OK;
}
