// Dense attention over 4-bit caches (dense_attn_q4 in lidx.h).
#include "q4.cuh"

namespace lidx {
namespace {

size_t split_bytes(int64_t n_rows, int Hq, int dv) { return (size_t)n_rows * Hq * (dv + 2) * sizeof(float); }

}  // namespace

size_t q4_attn_workspace_bytes(int dtype, int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv, int dk, int dv) {
    const int splits = dense_generic_splits(n_seq, n_q, max_n_kv, Hq, Hkv, dk, dv);
    return splits > kDenseCluster ? splits * split_bytes(n_seq * n_q, Hq, dv) : 0;
}

cudaError_t launch_attn_q4(DenseArgs a, int dtype, const Geom& g, void* ws, size_t ws_bytes, cudaStream_t st) {
    const int64_t n_rows = (int64_t)g.B * g.T;
    const int64_t fit = (int64_t)(ws_bytes / split_bytes(n_rows, a.Hq, a.dv));
    int64_t splits = dense_generic_splits(g.B, g.T, g.max_n_kv, a.Hq, a.Hkv, a.dk, a.dv);
    if (splits > kDenseCluster && splits > fit) splits = fit > kDenseCluster ? fit : kDenseCluster;
    a.splits = (int32_t)(splits < 1 ? 1 : splits);
    const bool apart = splits > kDenseCluster;
    a.part_o = apart ? static_cast<float*>(ws) : nullptr;
    a.part_ml = apart ? a.part_o + (size_t)n_rows * a.Hq * a.dv * splits : nullptr;
    cudaError_t e = launch_dense_generic_q4(a, dtype, g, st);
    if (e == cudaSuccess && apart) e = launch_dense_combine(a, dtype, n_rows, st);
    return e;
}

}  // namespace lidx
