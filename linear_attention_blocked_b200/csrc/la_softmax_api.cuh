// la_softmax_api.cuh -- C entry points of the softmax-attention operators and
// the paged key/value cache: argument checks, workspaces, tensor maps and
// launches.  Part of la_lib.cu (uses its helpers and status word).
#pragma once

namespace {

SmemAttr g_attr_softmax;

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

la_status check_softmax(int H, int Hkv, int d, float scale) {
    if (H <= 0 || Hkv <= 0 || d <= 0 || H % Hkv) return LA_ERR_INVALID_ARGUMENT;
    if (!(scale > 0.f) || scale > 3.0e38f) return LA_ERR_INVALID_ARGUMENT;  // also rejects NaN
    if (d != la::D) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

constexpr float kLog2e = 1.44269504088896341f;

int *status_word() {
    int *status = nullptr;
    if (cudaGetSymbolAddress(reinterpret_cast<void **>(&status), g_la_status) != cudaSuccess) return nullptr;
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

struct PagedCache {
    void *k, *v;
    int n_pages, page;
    const int *table;
    int max_pages;
    const int *lens;
};

la_status softmax_prefill_impl(const void *q, const void *k, const void *v, const int *cu, int nseq, long long T,
                               int max_seqlen, int H, int Hkv, int d, float scale, void *out, float *lse,
                               void *workspace, size_t ws_bytes, cudaStream_t stream) {
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
    const size_t n_q = (size_t)T * H * la::D * 2, n_kv = (size_t)T * Hkv * la::D * 2, n_lse = (size_t)T * H * 4;
    if (ranges_overlap(out, n_q, q, n_q) || ranges_overlap(out, n_q, k, n_kv) || ranges_overlap(out, n_q, v, n_kv) ||
        ranges_overlap(lse, n_lse, q, n_q) || ranges_overlap(lse, n_lse, k, n_kv) ||
        ranges_overlap(lse, n_lse, v, n_kv) || ranges_overlap(lse, n_lse, out, n_q))
        return LA_ERR_INVALID_ARGUMENT;
    const SoftmaxLayout w = softmax_layout(nseq, T);
    if (!workspace || ws_bytes < w.total) return LA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return LA_ERR_INVALID_ARGUMENT;
    if (ranges_overlap(workspace, w.total, out, n_q) || ranges_overlap(workspace, w.total, lse, n_lse))
        return LA_ERR_INVALID_ARGUMENT;
    const int G = H / Hkv, rows = G % 2 ? 2 * la::BLK : la::BLK, pairs = G % 2 ? G : G / 2;
    if (w.emax * Hkv * (long long)pairs > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    int *status = status_word();
    if (!status) return LA_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);

    la::SoftmaxScheduleParams sp;
    sp.cu = cu;
    sp.past = nullptr;
    sp.nseq = nseq;
    sp.T = (int)T;
    sp.max_seqlen = max_seqlen;
    sp.max_keys = 0;
    sp.rows = rows;
    sp.items_per_entry = Hkv * pairs;
    sp.hdr = reinterpret_cast<int *>(ws + w.hdr);
    sp.prefix = reinterpret_cast<int *>(ws + w.prefix);
    sp.entries = reinterpret_cast<int4 *>(ws + w.entries);
    sp.status = status;
    la::la_softmax_schedule_kernel<<<1, la::SCHED_THREADS, 0, stream>>>(sp);
    if (cudaGetLastError() != cudaSuccess) return LA_ERR_CUDA;
    ++g_launches;
    if (T == 0) return LA_OK;

    CUtensorMap mq, mk, mv;
    if (!encode_qkv_map(&mq, q, (int)T, H) || !encode_qkv_map(&mk, k, (int)T, Hkv) ||
        !encode_qkv_map(&mv, v, (int)T, Hkv))
        return LA_ERR_CUDA;
    la::SoftmaxPrefillParams pp;
    memset(&pp, 0, sizeof pp);
    pp.out = static_cast<__nv_bfloat16 *>(out);
    pp.lse = lse;
    pp.hdr = sp.hdr;
    pp.entries = sp.entries;
    pp.H = H;
    pp.Hkv = Hkv;
    pp.G = G;
    pp.pairs = pairs;
    pp.rows = rows;
    pp.scale_log2 = scale * kLog2e;
    pp.wait_limit_ns = g_wait_limit_ns.load();
    pp.status = status;
    const long long items = w.emax * Hkv * (long long)pairs;
    const int grid = (int)(items < device_sm_count() ? items : device_sm_count());
    st = ensure_smem_attr(g_attr_softmax, la::la_softmax_prefill_kernel, la::SMX_SMEM);
    if (st != LA_OK) return st;
    la::la_softmax_prefill_kernel<<<grid, la::SMX_THREADS, la::SMX_SMEM, stream>>>(mq, mk, mv, pp);
    if (cudaGetLastError() != cudaSuccess) return LA_ERR_CUDA;
    ++g_launches;
    return LA_OK;
}

}  // namespace

size_t la_softmax_prefill_varlen_workspace_size(int nseq, int total_tokens, int H, int Hkv, int d) {
    if (nseq < 0 || total_tokens < 0 || check_softmax(H, Hkv, d, 1.f) != LA_OK) return 0;
    return softmax_layout(nseq, total_tokens).total;
}

la_status la_softmax_prefill_varlen(const void *q, const void *k, const void *v, const int *cu_seqlens, int nseq,
                                    int total_tokens, int max_seqlen, int H, int Hkv, int d, float scale, void *out,
                                    float *lse, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    return softmax_prefill_impl(q, k, v, cu_seqlens, nseq, total_tokens, max_seqlen, H, Hkv, d, scale, out, lse,
                                workspace, ws_bytes, stream);
}
