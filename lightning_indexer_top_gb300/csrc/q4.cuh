// Rows of 4-bit caches, and the rows of new tokens (see "4-bit caches" and idx_new_rows in lidx.h).
#pragma once

#include "dense_attn.cuh"

namespace lidx {

// bytes of n heads of d columns: codes, then scale and minimum of each head
inline int64_t q4_payload(int64_t n, int64_t d) { return n * (d / 2 + 8); }

struct AppendArgs {
    idx_new_rows rows;
    int32_t Hq, Hkv, dk, dv;
    const float* inv_freq;
    int32_t n_rot, start, interleaved;
    void* k_cache;
    void* v_cache;
    int64_t kc_stride, vc_stride;    // elements; 4-bit caches: bytes
    int64_t kv_rows;
    int32_t k_lanes, v_lanes;        // lanes of a head row that is quantised from registers, 0: through shared memory (set by the launch)
};

cudaError_t launch_append(const AppendArgs& a, int dtype, bool q4, const Geom& g, cudaStream_t st);

struct ReadArgs {
    const void* k_cache;
    const void* v_cache;             // or NULL
    int64_t kc_stride, vc_stride;    // bytes
    int64_t kv_rows;
    int32_t Hkv, dk, dv;
    void* k_out;
    void* v_out;
};

cudaError_t launch_read_q4(const ReadArgs& a, int dtype, const Geom& g, cudaStream_t st);

// The positions of each sequence's span (device, [lo, hi)) for the attention: the values of K in dtype, row b * g.T + position,
// what they lack of their f32 in k_rest, and V in f16 (and v_rest).  A position whose cache row is out of range, with a number of K beyond
// dtype's, or with numbers that the powers of two leave too few bits sets *lost, in place of the device status.
struct ExpandArgs {
    ReadArgs r;
    const int2* span;
    int* lost;
    void* k_rest;
    void* v_rest;          // or NULL.  What V lacks
    const int* v_top;      // [B, Hkv]: V becomes f16 times 2^-v_exponent of this
    const int* k_top;      // or NULL.  Likewise K, by k_exponent
};

cudaError_t launch_expand_q4(const ExpandArgs& a, int dtype, const Geom& g, cudaStream_t st);

// dense_attn_q4 of checked arguments (k and v of a: bytes, strides in bytes)
cudaError_t launch_attn_q4(DenseArgs a, int dtype, const Geom& g, void* ws, size_t ws_bytes, cudaStream_t st);
size_t q4_attn_workspace_bytes(int dtype, int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv, int dk, int dv);

// cache row of batch row r (sequence b, token t), -1: none (*flagged: for a reason to report); *pos: its position
__device__ __forceinline__ int64_t new_row(const Geom& g, int64_t kv_rows, int64_t r, int b, int t, int* pos, bool* flagged) {
    const int n_kv = seq_n_kv(g, b);
    const int p = g.q_pos ? g.q_pos[r] : n_kv - g.T + t;
    *pos = p;
    *flagged = false;
    if (p < 0) return -1;
    int64_t row = -1;
    if (p < n_kv) row = key_row(g, b, p);
    if (row < 0 || row >= kv_rows) {
        *flagged = true;
        return -1;
    }
    return row;
}

}  // namespace lidx
