// What the dense attention kernels share: the options, a row's interval of
// visible keys, and the partial results of key splits.
#pragma once

#include "lidx_internal.cuh"
#include "sm100_ptx.cuh"

namespace lidx {

constexpr int kDenseMaxSplits = 128;   // key splits, at most (the merge keeps their weights in a warp)

constexpr int kDenseCluster = 8;       // splits that a cluster merges itself, at most

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
    int32_t splits;           // key splits; > 1: partial results go to part_o / part_ml, or, without those (at most
                              // kDenseCluster splits), the splits are a cluster that merges them
    float* part_o;            // [row * Hq + head][split][dv] unnormalised
    float* part_ml;           // [row * Hq + head][split][2]: maximum (natural-log units), sum
    const void* k_rest;       // or NULL.  Given (tensor cores): K is the sum of k and this, laid out alike, and V f16
    const int* v_top;         // ... at the power of two that v_exponent makes of this [B, Hkv]
    const void* v_rest;       // ... with f16 q: what V lacks of its f32, in f16, laid out alike; K is at the power of two that
                              // k_exponent makes of another [B, Hkv] behind v_top then
    const int* only_if;       // or NULL; given and 0 on the device: the launch has nothing to do (CUDA cores, 4 bits)
};

// The power of two at which f16 holds numbers of magnitudes up to top (a float's bits) as numbers below 2^15, so that those
// 2^28 below the largest keep f16's eleven bits: -126 .. 113; and 2^n, n in [-126, 127]
__device__ __forceinline__ int v_exponent(int top) { return max((top >> 23) - 127, -112) - 14; }

// The same for K, whose power goes with the call's scale (so it is no smaller than 2^-60)
__device__ __forceinline__ int k_exponent(int top) { return max(v_exponent(top), -60); }

__device__ __forceinline__ float exp2_whole(int n) { return __int_as_float((n + 127) << 23); }

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
            if (m.prefix_end) h = max(h, m.prefix_end[r]);
            v.hi = min(n_kv, h);
            if (m.window > 0) v.lo = max(0, p - m.window + 1);
        }
    }
    if (m.doc_start) v.lo = max(v.lo, m.doc_start[r]);
    return v;
}

// rows per TMA box of a tile of `keys` positions: all of them, or the largest power of two that divides the page
inline int box_rows(int page_size, int keys) {
    if (!page_size) return keys;
    const int b = page_size & -page_size;
    return b < keys ? b : keys;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// the options as the softmax applies them, in log2 units
struct Score {
    float c;            // scale * log2(e)
    float inv_cap;      // scale / softcap (0: no cap)
    float cap;          // softcap * log2(e)
    float series;       // the largest product whose capped score is the series in it; below 0: none is
    float slope;        // the row's slope * log2(e)
    bool biased;        // slopes are given
};

// two f32 in one 64-bit register, for the packed FMA and add
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 1 - 2 / (1 + e^(2x)): for |x| > 0.3, where it does not cancel
__device__ __forceinline__ float tanh_large(float x) {
    return fmaf(-2.f, rcp_approx(1.f + sm100::ex2_approx(x * (2.f * kLog2e))), 1.f);
}

// N raw products of consecutive keys -> scores in log2 units; d0 = the row's position minus the first key's; past:
// no key that the warp's rows see lies past their positions (no absolute value to take, one operation less).
// Every lane of a warp comes here together.
// A capped score is cap * tanh(x), x = s * scale / softcap: for |x| <= 0.3 by the Taylor series of tanh up to x^9
// (the next term is below 2^-24 of x there), as s times a polynomial in s^2 whose coefficients hold the factors (six
// packed operations for two scores; the exponential form takes two special functions for each).  Where those
// coefficients, scale * (scale / softcap)^8 the farthest, leave f32's normal range, the series is taken in x itself.
template <int N>
__device__ __forceinline__ void modify(float (&s)[N], const Score& sc, float d0, bool past) {
    if (sc.inv_cap != 0.f) {
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < N; i += 2) big = fmaxf(fmaxf(big, fabsf(s[i])), fabsf(s[i + 1]));
        const float i2 = sc.inv_cap * sc.inv_cap;
        // (a NaN is no larger than anything and goes through the series)
        const bool large = big > sc.series;
        auto both = [](float x) { return pair(x, x); };
        const uint64_t c1 = both(sc.c), c3 = both(sc.c * i2 * (-1.f / 3.f)), c5 = both(sc.c * i2 * i2 * (2.f / 15.f)),
                       c7 = both(sc.c * i2 * i2 * i2 * (-17.f / 315.f)),
                       c9 = both(sc.c * i2 * i2 * i2 * i2 * (62.f / 2835.f));
        // (the x^9 term is below 2^-27 of x up to 0.15)
        const bool some = big > 0.5f * sc.series;
        if (__any_sync(0xffffffffu, large)) {
            const uint64_t inv = both(sc.inv_cap), one = both(1.f);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const uint64_t v = pair(s[i], s[i + 1]), x = mul2(v, inv), z = mul2(x, x);
                const uint64_t p = fma2(fma2(fma2(fma2(both(62.f / 2835.f), z, both(-17.f / 315.f)), z, both(2.f / 15.f)), z,
                                             both(-1.f / 3.f)), z, one);
                float x0, x1, y0, y1;
                unpair(x, x0, x1);
                unpair(mul2(mul2(v, c1), p), y0, y1);
                s[i] = fabsf(x0) > 0.3f ? sc.cap * tanh_large(x0) : y0;
                s[i + 1] = fabsf(x1) > 0.3f ? sc.cap * tanh_large(x1) : y1;
            }
        } else if (__any_sync(0xffffffffu, some)) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const uint64_t v = pair(s[i], s[i + 1]), z = mul2(v, v);
                unpair(mul2(v, fma2(fma2(fma2(fma2(c9, z, c7), z, c5), z, c3), z, c1)), s[i], s[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const uint64_t v = pair(s[i], s[i + 1]), z = mul2(v, v);
                unpair(mul2(v, fma2(fma2(fma2(c7, z, c5), z, c3), z, c1)), s[i], s[i + 1]);
            }
        }
    } else {
        const uint64_t c = pair(sc.c, sc.c);
#pragma unroll
        for (int i = 0; i < N; i += 2) unpair(mul2(pair(s[i], s[i + 1]), c), s[i], s[i + 1]);
    }
    if (sc.biased) {
        if (past) {
            const uint64_t sl = pair(sc.slope, sc.slope), base = pair(-sc.slope * d0, -sc.slope * d0);
#pragma unroll
            for (int i = 0; i < N; i += 2)
                unpair(add2(pair(s[i], s[i + 1]), fma2(sl, pair((float)i, (float)(i + 1)), base)), s[i], s[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = fmaf(-sc.slope, fabsf(d0 - (float)i), s[i]);
        }
    }
}

// scale: a.scale, times the power of two at which K is
__device__ __forceinline__ Score make_score(const DenseArgs& a, float scale, float slope) {
    Score s;
    s.c = scale * kLog2e;
    s.inv_cap = a.mods.softcap > 0.f ? scale / a.mods.softcap : 0.f;
    s.cap = a.mods.softcap * kLog2e;
    const float i2 = s.inv_cap * s.inv_cap, c9 = fabsf(s.c * i2 * i2 * i2 * i2 * (62.f / 2835.f));
    s.series = c9 >= 0x1p-126f && c9 <= 0x1p100f ? 0.3f / fabsf(s.inv_cap) : -1.f;
    s.slope = slope * kLog2e;
    s.biased = a.mods.slopes != nullptr;
    return s;
}

// CUDA cores: every type, width and alignment
cudaError_t launch_dense_generic(const DenseArgs& a, int dtype, const Geom& g, cudaStream_t st);
int dense_generic_splits(int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv, int dk, int dv);
// the same over 4-bit caches (k and v: bytes, strides in bytes; dk and dv multiples of 8)
cudaError_t launch_dense_generic_q4(const DenseArgs& a, int dtype, const Geom& g, cudaStream_t st);

// tensor cores: 16-bit K and V of at most 128 columns each, 16-byte aligned, pages of a multiple of 8 rows
bool dense_tc_supported(const DenseArgs& a, int dtype, const Geom& g);
cudaError_t launch_dense_tc(const DenseArgs& a, int dtype, const Geom& g, cudaStream_t st);
int dense_tc_splits(int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv);
constexpr int kDenseTcKeys = 128;   // its splits are whole tiles of this many keys

// tensor cores: the bf16 MLA latent of 128 heads (576 / 512 columns), 2-CTA clusters; its own key splits and partials
bool dense_mla_supported(const DenseArgs& a, int dtype, const Geom& g);
int dense_mla_splits(int64_t n_rows, int64_t max_n_kv);
size_t dense_mla_workspace_bytes(int64_t n_rows, int64_t max_n_kv);
cudaError_t launch_dense_mla(const DenseArgs& a, const Geom& g, void* ws, size_t ws_bytes, cudaStream_t st);

// merges part_o / part_ml into out and lse
cudaError_t launch_dense_combine(const DenseArgs& a, int dtype, int64_t n_rows, cudaStream_t st);

}  // namespace lidx
