// C-ABI entry points of the dense attention and of the page operations.
#include <stdarg.h>
#include <stdio.h>

#include <cmath>

#include "dense_attn.cuh"

namespace lidx {

size_t page_workspace_bytes(int64_t n_seq, int64_t n_pages);
bool page_caches_fit(const idx_page_cache* caches, int n, int page_size);
cudaError_t launch_page_copy(const idx_page_cache* caches, int n_caches, int page_size, int32_t n_pages,
                             const int32_t* src, const int32_t* dst, int32_t n, cudaStream_t st);
cudaError_t launch_page_update(const int32_t* table, int64_t stride, int32_t cols, int32_t n_old, const int32_t* parent,
                               const int32_t* keep, const int32_t* len, int32_t n_seq, int32_t ps, int32_t n_pages,
                               const uint8_t* held, int32_t* out, int64_t out_stride, int32_t out_cols,
                               int32_t* n_free, const idx_page_cache* caches, int n_caches, void* ws, cudaStream_t st);
cudaError_t launch_page_compact(const int32_t* table, int64_t stride, int32_t cols, int32_t n_seq, const int32_t* len,
                                int32_t ps, int32_t n_pages, const uint8_t* held, int32_t* out, int64_t out_stride,
                                int32_t* n_used, int32_t* remap, const idx_page_cache* caches, int n_caches, void* ws,
                                cudaStream_t st);

namespace {

idx_status bad(idx_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return record_error(s, buf);
}

// the key splits that a call of these sizes would like (the tensor-core kernel's where its types and widths are)
int want_splits(int dtype, int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv, int dk, int dv, bool tc) {
    return tc ? dense_tc_splits(n_seq, n_q, max_n_kv, Hq, Hkv)
              : dense_generic_splits(n_seq, n_q, max_n_kv, Hq, Hkv, dk, dv);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// bytes of one split's partial results
size_t split_bytes(int64_t n_rows, int Hq, int dv) { return (size_t)n_rows * Hq * (dv + 2) * sizeof(float); }

idx_status check_caches(const char* what, const idx_page_cache* caches, int32_t n, int32_t page_size, int32_t n_pages,
                        int32_t least) {
    if (n < least || n > IDX_MAX_PAGE_CACHES)
        return bad(IDX_ERR_INVALID_ARG, "%s: n_caches must be in [%d, %d]", what, least, IDX_MAX_PAGE_CACHES);
    if (page_size < 1) return bad(IDX_ERR_INVALID_ARG, "%s: page_size < 1", what);
    if (n_pages < 0) return bad(IDX_ERR_INVALID_ARG, "%s: n_pages < 0", what);
    if (n > 0 && !caches) return bad(IDX_ERR_INVALID_ARG, "%s: caches is NULL", what);
    for (int i = 0; i < n; ++i) {
        if (caches[i].row_bytes < 1 || caches[i].row_stride_bytes < caches[i].row_bytes)
            return bad(IDX_ERR_INVALID_ARG, "%s: cache %d: need 1 <= row_bytes <= row_stride_bytes", what, i);
        if (n_pages > 0 && !caches[i].data) return bad(IDX_ERR_INVALID_ARG, "%s: cache %d: data is NULL", what, i);
        if (caches[i].row_stride_bytes > INT64_MAX / page_size / (n_pages > 0 ? n_pages : 1))
            return bad(IDX_ERR_INVALID_ARG, "%s: cache %d: larger than the address space", what, i);
    }
    if (!page_caches_fit(caches, n, page_size)) return bad(IDX_ERR_UNSUPPORTED, "%s: pages too large", what);
    return IDX_OK;
}

}  // namespace
}  // namespace lidx

using namespace lidx;

extern "C" {

size_t dense_attn_workspace_size(idx_dtype dtype, int32_t n_seq, int32_t n_q_per_seq, int32_t max_n_kv,
                                 int32_t n_q_heads, int32_t n_kv_heads, int32_t dk, int32_t dv) {
    if (n_seq < 1 || n_q_per_seq < 1 || max_n_kv < 1 || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads ||
        dk < 1 || dk > 576 || dv < 1 || dv > 512)
        return 0;
    if (dtype == IDX_BF16 && n_q_heads == 128 && n_kv_heads == 1 && dk == 576 && dv == 512)
        return dense_mla_workspace_bytes((int64_t)n_seq * n_q_per_seq, max_n_kv);
    // (a call whose pages or addresses the tensor-core kernel does not take splits as far as this reaches)
    const bool tc = dtype != IDX_F32 && dk <= 128 && dv <= 128 && dk % 8 == 0 && dv % 8 == 0;
    const int splits = want_splits(dtype, n_seq, n_q_per_seq, max_n_kv, n_q_heads, n_kv_heads, dk, dv, tc);
    return splits > kDenseCluster ? splits * split_bytes((int64_t)n_seq * n_q_per_seq, n_q_heads, dv) : 0;
}

idx_status dense_attn(const void* q, idx_dtype dtype, int32_t n_q_heads, int32_t n_kv_heads, int32_t dk, int32_t dv,
                      const void* k, const void* v, int64_t kv_row_stride, int64_t v_row_stride, int64_t kv_rows,
                      idx_batch batch, const idx_attn_mods* mods, float scale, void* out, float* lse,
                      void* workspace, size_t workspace_bytes, idx_stream_t stream) {
    const char* what = "dense_attn";
    idx_status s = validate_batch(batch, what);
    if (s != IDX_OK) return s;
    if (dtype != IDX_F32 && dtype != IDX_F16 && dtype != IDX_BF16)
        return bad(IDX_ERR_INVALID_ARG, "%s: bad dtype", what);
    if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads != 0)
        return bad(IDX_ERR_INVALID_ARG, "%s: need Hq, Hkv >= 1 and Hq %% Hkv == 0", what);
    if (dk < 1 || dk > 576 || dv < 1 || dv > 512)
        return bad(IDX_ERR_INVALID_ARG, "%s: need 1 <= dk <= 576 and 1 <= dv <= 512", what);
    if (!v && (n_kv_heads != 1 || dv > dk))
        return bad(IDX_ERR_INVALID_ARG, "%s: latent form (v == NULL) needs Hkv == 1, dv <= dk", what);
    if (kv_row_stride < (int64_t)n_kv_heads * dk) return bad(IDX_ERR_INVALID_ARG, "%s: kv_row_stride < Hkv*dk", what);
    if (v && v_row_stride < (int64_t)n_kv_heads * dv)
        return bad(IDX_ERR_INVALID_ARG, "%s: v_row_stride < Hkv*dv", what);
    if (kv_rows < 0) return bad(IDX_ERR_INVALID_ARG, "%s: kv_rows < 0", what);
    // (the tensor-core kernels hold both times log2(e))
    if (!(std::fabs(scale) <= 0x1p127f)) return bad(IDX_ERR_INVALID_ARG, "%s: scale not finite or above 2^127", what);
    DenseArgs a = {};
    if (mods) a.mods = *mods;
    if (!(a.mods.softcap >= 0.f && a.mods.softcap <= 0x1p127f))
        return bad(IDX_ERR_INVALID_ARG, "%s: softcap must be finite and >= 0, at most 2^127", what);
    if (a.mods.softcap > 0.f && !std::isfinite(scale / a.mods.softcap))
        return bad(IDX_ERR_INVALID_ARG, "%s: scale / softcap must be finite", what);
    if (a.mods.window < 0) return bad(IDX_ERR_INVALID_ARG, "%s: window < 0", what);
    if (!batch.q_pos && (a.mods.window > 0 || a.mods.slopes || a.mods.prefix_len || a.mods.prefix_end))
        return bad(IDX_ERR_INVALID_ARG, "%s: window, slopes, prefix_len and prefix_end need q_pos", what);
    if (workspace && !aligned16(workspace))
        return bad(IDX_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", what);
    if (batch.max_n_kv > INT32_MAX - 1024)
        return bad(IDX_ERR_UNSUPPORTED, "%s: max_n_kv must be at most 2^31 - 1025", what);
    const int64_t n_rows = (int64_t)batch.n_seq * batch.n_q_per_seq;
    if (n_rows == 0) return IDX_OK;
    if (!q || !out || (batch.max_n_kv > 0 && !k)) return bad(IDX_ERR_INVALID_ARG, "%s: NULL q/k/out", what);
    a.q = q;
    a.Hq = n_q_heads;
    a.Hkv = n_kv_heads;
    a.dk = dk;
    a.dv = dv;
    a.k = k;
    a.v = v;
    a.k_stride = kv_row_stride;
    a.v_stride = v_row_stride;
    a.kv_rows = kv_rows;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    const Geom g = geom_of(batch);
    const cudaStream_t st = (cudaStream_t)stream;
    if (dense_mla_supported(a, dtype, g)) {
        const cudaError_t e = launch_dense_mla(a, g, workspace, workspace ? workspace_bytes : 0, st);
        if (e != cudaErrorNotSupported) return cuda_status(e, what);
    }
    const size_t per_split = split_bytes(n_rows, n_q_heads, dv);
    const int64_t fit = workspace ? (int64_t)(workspace_bytes / per_split) : 0;
    const bool tc = dense_tc_supported(a, dtype, g);
    int64_t splits = want_splits(dtype, batch.n_seq, batch.n_q_per_seq, batch.max_n_kv, n_q_heads, n_kv_heads, dk, dv, tc);
    // up to kDenseCluster splits are a cluster and need no workspace
    if (splits > kDenseCluster && splits > fit) splits = fit > kDenseCluster ? fit : kDenseCluster;
    // a split gets whole tiles of the keys that its rows see: no more splits than tiles
    const int64_t tiles = ((int64_t)batch.max_n_kv + (tc ? kDenseTcKeys : 1) - 1) / (tc ? kDenseTcKeys : 1);
    if (splits > tiles) splits = tiles;
    if (splits < 1) splits = 1;
    a.splits = (int32_t)splits;
    const bool apart = splits > kDenseCluster;
    a.part_o = apart ? static_cast<float*>(workspace) : nullptr;
    a.part_ml = apart ? a.part_o + (size_t)n_rows * n_q_heads * dv * splits : nullptr;
    cudaError_t e = tc ? launch_dense_tc(a, dtype, g, st) : cudaErrorNotSupported;
    if (e == cudaErrorNotSupported) e = launch_dense_generic(a, dtype, g, st);
    if (e == cudaSuccess && apart) e = launch_dense_combine(a, dtype, n_rows, st);
    return cuda_status(e, what);
}

size_t idx_page_workspace_size(int32_t n_seq, int32_t n_pages) {
    return n_seq < 0 || n_pages < 0 ? 0 : page_workspace_bytes(n_seq, n_pages);
}

idx_status idx_page_copy(const idx_page_cache* caches, int32_t n_caches, int32_t page_size, int32_t n_pages,
                         const int32_t* src, const int32_t* dst, int32_t n, idx_stream_t stream) {
    const char* what = "idx_page_copy";
    const idx_status s = check_caches(what, caches, n_caches, page_size, n_pages, 1);
    if (s != IDX_OK) return s;
    if (n < 0) return bad(IDX_ERR_INVALID_ARG, "%s: n < 0", what);
    if (n == 0) return IDX_OK;
    if (!src || !dst) return bad(IDX_ERR_INVALID_ARG, "%s: NULL src/dst", what);
    return cuda_status(launch_page_copy(caches, n_caches, page_size, n_pages, src, dst, n, (cudaStream_t)stream), what);
}

idx_status idx_page_update(const int32_t* page_table, int64_t table_stride, int32_t table_cols, int32_t n_seq_old,
                           const int32_t* parent, const int32_t* n_keep, const int32_t* n_new, int32_t n_seq,
                           int32_t page_size, int32_t n_pages, const uint8_t* held, int32_t* new_table,
                           int64_t new_stride, int32_t new_cols, int32_t* n_free, const idx_page_cache* caches,
                           int32_t n_caches, void* workspace, size_t workspace_bytes, idx_stream_t stream) {
    const char* what = "idx_page_update";
    const idx_status s = check_caches(what, caches, n_caches, page_size, n_pages, 0);
    if (s != IDX_OK) return s;
    if (n_seq_old < 0 || n_seq < 0) return bad(IDX_ERR_INVALID_ARG, "%s: n_seq_old or n_seq < 0", what);
    if (table_cols < 0 || new_cols < 0 || table_stride < table_cols || new_stride < new_cols)
        return bad(IDX_ERR_INVALID_ARG, "%s: need 0 <= columns <= stride for both tables", what);
    if ((int64_t)n_seq * new_cols > INT32_MAX || (int64_t)n_seq_old * table_cols > INT32_MAX)
        return bad(IDX_ERR_INVALID_ARG, "%s: more than 2^31-1 table entries", what);
    if (!n_free || (n_seq > 0 && (!parent || !n_keep || !n_new || (new_cols > 0 && !new_table))) ||
        (n_seq_old > 0 && table_cols > 0 && !page_table))
        return bad(IDX_ERR_INVALID_ARG, "%s: NULL page_table/parent/n_keep/n_new/new_table/n_free", what);
    if (n_seq > 0 && new_cols > 0 && n_seq_old > 0 && table_cols > 0) {
        const int32_t* o1 = page_table + (n_seq_old - 1) * table_stride + table_cols;
        const int32_t* w1 = new_table + (n_seq - 1) * new_stride + new_cols;
        if (page_table < w1 && new_table < o1) return bad(IDX_ERR_INVALID_ARG, "%s: new_table overlaps page_table", what);
    }
    const size_t need = idx_page_workspace_size(n_seq, n_pages);
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
        return bad(IDX_ERR_INVALID_ARG, "%s: needs a 16-byte aligned workspace of %zu bytes (idx_page_workspace_size)",
                   what, need);
    return cuda_status(launch_page_update(page_table, table_stride, table_cols, n_seq_old, parent, n_keep, n_new, n_seq,
                                          page_size, n_pages, held, new_table, new_stride, new_cols, n_free, caches,
                                          n_caches, workspace, (cudaStream_t)stream),
                       what);
}

idx_status idx_page_compact(const int32_t* page_table, int64_t table_stride, int32_t table_cols, int32_t n_seq,
                            const int32_t* n_len, int32_t page_size, int32_t n_pages, const uint8_t* held,
                            int32_t* new_table, int64_t new_stride, int32_t* n_used, int32_t* remap,
                            const idx_page_cache* caches, int32_t n_caches, void* workspace, size_t workspace_bytes,
                            idx_stream_t stream) {
    const char* what = "idx_page_compact";
    const idx_status s = check_caches(what, caches, n_caches, page_size, n_pages, 0);
    if (s != IDX_OK) return s;
    if (n_seq < 0) return bad(IDX_ERR_INVALID_ARG, "%s: n_seq < 0", what);
    if (table_cols < 0 || table_stride < table_cols || new_stride < table_cols)
        return bad(IDX_ERR_INVALID_ARG, "%s: need 0 <= table_cols <= both strides", what);
    if ((int64_t)n_seq * table_cols > INT32_MAX)
        return bad(IDX_ERR_INVALID_ARG, "%s: more than 2^31-1 table entries", what);
    if (!n_used || (n_seq > 0 && (!n_len || (table_cols > 0 && (!page_table || !new_table)))))
        return bad(IDX_ERR_INVALID_ARG, "%s: NULL page_table/n_len/new_table/n_used", what);
    if (n_seq > 0 && table_cols > 0) {
        const int32_t* o1 = page_table + (n_seq - 1) * table_stride + table_cols;
        const int32_t* w1 = new_table + (n_seq - 1) * new_stride + table_cols;
        const bool same = new_table == page_table && new_stride == table_stride;
        if (!same && page_table < w1 && new_table < o1)
            return bad(IDX_ERR_INVALID_ARG, "%s: new_table overlaps page_table without being it", what);
    }
    const size_t need = idx_page_workspace_size(n_seq, n_pages);
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
        return bad(IDX_ERR_INVALID_ARG, "%s: needs a 16-byte aligned workspace of %zu bytes (idx_page_workspace_size)",
                   what, need);
    return cuda_status(launch_page_compact(page_table, table_stride, table_cols, n_seq, n_len, page_size, n_pages, held,
                                           new_table, new_stride, n_used, remap, caches, n_caches, workspace,
                                           (cudaStream_t)stream),
                       what);
}

}  // extern "C"
