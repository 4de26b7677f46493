// What the dense attention kernels share: the options, a row's interval of
// visible keys, and the partial results of key splits.
#pragma once

#include "lidx_internal.cuh"

namespace lidx {

struct DenseArgs {
    const void* q;
    int32_t Hq, Hkv, dk, dv;
    const void* k;
    const void* v;            // NULL: the first dv columns of the K row
    int64_t k_stride, v_stride;
    int64_t kv_rows;
    float scale;
    idx_attn_mods mods;
    void* out;                // of q's type
    float* lse;               // or NULL
    int32_t splits;           // key splits; > 1: partial results go to part_o / part_ml
    int32_t kps;              // keys of the position line per split
    float* part_o;            // [row * Hq + head][split][dv] unnormalised
    float* part_ml;           // [row * Hq + head][split][2]: maximum (natural-log units), sum
};

struct Interval {
    int lo, hi;               // visible positions [lo, hi); lo >= hi: none
    int pos;                  // the row's own position (0 without q_pos)
};

// n_kv: the sequence's cached tokens (seq_n_kv)
__device__ __forceinline__ Interval row_interval(const Geom& g, const idx_attn_mods& m, int64_t r, int b, int n_kv) {
    Interval v;
    v.pos = 0;
    v.lo = 0;
    v.hi = n_kv;
    if (g.q_pos) {
        const int p = g.q_pos[r];
        v.pos = p;
        if (p < 0) {
            v.hi = 0;
        } else {
            int h = p < INT32_MAX ? p + 1 : p;
            if (m.prefix_len) h = max(h, m.prefix_len[b]);
            v.hi = min(n_kv, h);
            if (m.window > 0) v.lo = max(0, p - m.window + 1);
        }
    }
    if (m.doc_start) v.lo = max(v.lo, m.doc_start[r]);
    return v;
}

// CUDA cores: every type, width and alignment
cudaError_t launch_dense_generic(const DenseArgs& a, int dtype, const Geom& g, cudaStream_t st);
int dense_generic_splits(int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv, int dk, int dv);

// tensor cores: 16-bit K and V of at most 128 columns each, 16-byte aligned, pages of a multiple of 8 rows
bool dense_tc_supported(const DenseArgs& a, int dtype, const Geom& g);
cudaError_t launch_dense_tc(const DenseArgs& a, int dtype, const Geom& g, cudaStream_t st);
int dense_tc_splits(int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv);
constexpr int kDenseTcKeys = 128;   // its splits are whole tiles of this many keys

// merges part_o / part_ml into out and lse
cudaError_t launch_dense_combine(const DenseArgs& a, int dtype, int64_t n_rows, cudaStream_t st);

}  // namespace lidx
