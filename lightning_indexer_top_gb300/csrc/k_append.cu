// Rows of new tokens into (paged) caches with the position rotation on the way,
// also into 4-bit caches, and the way back (idx_cache_append, idx_cache_append_q4
// and idx_cache_read_q4 in lidx.h).
//
// Rotation: pair i of a head's row at position p is turned by p * f[i].  f / 2 pi is
// taken as a 64-bit fraction of a turn u, so that p * u modulo 2^64 is the angle
// modulo a turn, exactly what far positions need: an f32 product p * f is off by
// 0.004 rad at position 65536.  Its top 32 bits go through sincospi in f32.
//
// A CTA owns a few tokens: one thread per (token, pair) makes cosine and sine once for
// every head, then the threads share the head rows in 16-byte pieces (a pair of
// pieces where the two halves of a rotation lie apart); odd widths, starts and
// alignments go element by element.  The bytes moved bound long chunks, launch and
// latency the rows of one decode step.
#include <float.h>

#include "q4.cuh"

namespace lidx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 8;      // per CTA
constexpr int kMaxD = 576;

// phase of position p in turns of 2^64
__device__ __forceinline__ uint64_t phase(float f, int p) {
    const double turns = (double)f * 0.15915494309189533577;     // 1 / 2 pi
    const double part = turns - floor(turns);
    return (uint64_t)(part * 18446744073709551616.0) * (uint64_t)(uint32_t)p;     // (a part of 1 saturates)
}

__device__ __forceinline__ float2 cos_sin(float f, int p) {
    const int32_t top = (int32_t)(uint32_t)(phase(f, p) >> 32);
    float s, c;
    sincospif((float)top * 0x1p-31f, &s, &c);
    return make_float2(c, s);
}

template <typename T, int E>
struct Piece {
    T x[E];
};

template <typename T, int E>
__device__ __forceinline__ Piece<T, E> load(const T* p) {
    Piece<T, E> v;
    if constexpr (E * sizeof(T) == 16)
        *reinterpret_cast<uint4*>(&v) = *reinterpret_cast<const uint4*>(p);
    else
        v.x[0] = *p;
    return v;
}

template <typename T, int E>
__device__ __forceinline__ void store(T* p, const Piece<T, E>& v) {
    if constexpr (E * sizeof(T) == 16)
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&v);
    else
        *p = v.x[0];
}

// a token's rows: where they come from, where they go
struct Token {
    int64_t row;      // batch row
    int64_t to;       // cache row, -1: none
    int pos;          // < 0: padding
};

// Unit u of a head row of w columns (rot: rotated): with the pairs apart, first the n_rot / 2 / E pairs of pieces, then the
// columns that stay; with the pairs side by side, pieces of E columns.
template <typename T, int E, bool kInter>
__device__ __forceinline__ void head_unit(const AppendArgs& a, const T* src, T* dst, int u, bool rot, const float2* cs) {
    const int n = rot ? a.n_rot : 0;
    if (kInter && E > 1) {
        const int c = u * E;
        Piece<T, E> v = load<T, E>(src + c);
        if (c >= a.start && c < a.start + n) {
            const float2* t = cs + (c - a.start) / 2;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float x = to_f32(v.x[2 * i]), y = to_f32(v.x[2 * i + 1]);
                v.x[2 * i] = from_f32<T>(fmaf(x, t[i].x, -(y * t[i].y)));
                v.x[2 * i + 1] = from_f32<T>(fmaf(y, t[i].x, x * t[i].y));
            }
        }
        store<T, E>(dst + c, v);
        return;
    }
    const int pairs = n / (2 * E);
    if (u < pairs) {
        const int c0 = kInter ? a.start + 2 * u : a.start + u * E, c1 = kInter ? c0 + 1 : c0 + n / 2;
        Piece<T, E> v = load<T, E>(src + c0), w = load<T, E>(src + c1);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float2 t = cs[u * E + i];
            const float x = to_f32(v.x[i]), y = to_f32(w.x[i]);
            v.x[i] = from_f32<T>(fmaf(x, t.x, -(y * t.y)));
            w.x[i] = from_f32<T>(fmaf(y, t.x, x * t.y));
        }
        store<T, E>(dst + c0, v);
        store<T, E>(dst + c1, w);
    } else {
        int c = (u - pairs) * E;
        if (c >= a.start) c += n;
        store<T, E>(dst + c, load<T, E>(src + c));
    }
}

// units of a head row of w columns
template <int E, bool kInter>
__device__ __forceinline__ int head_units(const AppendArgs& a, int w, bool rot) {
    return kInter && E > 1 ? w / E : rot ? (w - a.n_rot / 2) / E : w / E;
}

// ------------------------------------------------------------------------------------------- 4 bits

// column c of a head row after the rotation in 64 bits
template <typename T>
__device__ __forceinline__ double exact_column(const AppendArgs& a, const T* src, int c, bool rot, int p) {
    const double x = (double)to_f32(src[c]);
    if (!rot || p < 0 || c < a.start || c >= a.start + a.n_rot) return x;
    const int i = c - a.start, half = a.n_rot / 2;
    const bool second = a.interleaved ? i & 1 : i >= half;
    const int pr = a.interleaved ? i >> 1 : second ? i - half : i;
    const double y = (double)to_f32(src[a.interleaved ? a.start + (i ^ 1) : second ? c - half : c + half]);
    double s, co;
    sincospi((double)(int64_t)phase(a.inv_freq[pr], p) * 0x1p-63, &s, &co);
    return second ? x * co + y * s : x * co - y * s;
}

// A warp's head row of w columns into 4 bits at `codes` and `pair`.
// Rotated in f32 a column is off by at most 1.25 * 2^-22 of its pair's |u| + |w| (the angle by pi * 2^-25, cosine and sine by
// an ulp, three roundings), so t = 15 (x - min) / (max - min) by at most 60 such errors over max - min, and 15 * 2^-22 for
// its own roundings.  A row with a column that lies nearer than that to a border between codes is done again in 64 bits
// (one head row of 128 in about 200).
template <typename T>
__device__ __forceinline__ void quantize_row(const AppendArgs& a, const T* src, int w, bool rot, int p, const float2* cs,
                                             float* buf, uint8_t* codes, float* pair) {
    const int lane = threadIdx.x & 31;
    const int n = rot ? a.n_rot : 0, half = n / 2;
    float big = 0.f;       // the largest |u| + |w|
    float lo = INFINITY, hi = -INFINITY;
    bool fine = true;
    auto take = [&](int c, float y) {
        buf[c] = y;
        lo = fminf(lo, y);
        hi = fmaxf(hi, y);
        fine &= fabsf(y) <= FLT_MAX;
    };
    for (int i = lane; i < half; i += 32) {
        const int c0 = a.interleaved ? a.start + 2 * i : a.start + i, c1 = a.interleaved ? c0 + 1 : c0 + half;
        const float u = to_f32(src[c0]), v = to_f32(src[c1]);
        const float2 t = cs[i];
        big = fmaxf(big, fabsf(u) + fabsf(v));
        take(c0, fmaf(u, t.x, -(v * t.y)));
        take(c1, fmaf(v, t.x, u * t.y));
    }
    for (int i = lane; i < w - n; i += 32) {
        const int c = i < a.start || !n ? i : i + n;
        take(c, to_f32(src[c]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    }
    fine = __all_sync(0xffffffffu, fine);       // (and buf is written)
    const float span = hi - lo, inv = 15.f / span;
    const float eps = (60.f * 1.25f * 0x1p-22f) * big / span + 15.f * 0x1p-22f;
    // (a span of 0, or one whose inverse is no f32, is told apart below)
    bool sure = fine && inv <= FLT_MAX && inv > 0.f && span <= FLT_MAX && eps < 0.25f;
    bool same = fine && span == 0.f && !(big > 0.f);      // every column the same, exactly
    for (int word = lane; word - lane < w / 8; word += 32) {
        bool near = false;
        uint32_t x = 0u;
        if (word < w / 8 && sure) {
            const float4 y0 = *reinterpret_cast<const float4*>(buf + word * 8), y1 = *reinterpret_cast<const float4*>(buf + word * 8 + 4);
            const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = (y[i] - lo) * inv, r = rintf(t);
                near |= fabsf(t - r) > 0.5f - eps;
                x |= (uint32_t)(int)fminf(fmaxf(r, 0.f), 15.f) << (4 * i);
            }
        }
        sure = !__any_sync(0xffffffffu, near) && sure;
        if (!sure) break;
        if (word < w / 8) reinterpret_cast<uint32_t*>(codes)[word] = x;
    }
    float scale = span / 15.f, low = lo;
    if (!sure) {
        if (!fine) scale = low = __int_as_float(0x7fc00000);
        double dlo = 0.0, dspan = 0.0;
        if (fine && !same) {
            double a0 = INFINITY, a1 = -INFINITY;
            for (int c = lane; c < w; c += 32) {
                const double y = exact_column(a, src, c, rot, p);
                a0 = fmin(a0, y);
                a1 = fmax(a1, y);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                a0 = fmin(a0, __shfl_xor_sync(0xffffffffu, a0, o));
                a1 = fmax(a1, __shfl_xor_sync(0xffffffffu, a1, o));
            }
            dlo = a0;
            dspan = a1 - a0;
            scale = (float)(dspan / 15.0);
            low = (float)dlo;
        }
        __syncwarp();
        for (int c = lane; c < w; c += 32)
            buf[c] = dspan > 0.0 ? (float)rint((exact_column(a, src, c, rot, p) - dlo) * 15.0 / dspan) : 0.f;
        __syncwarp();
        for (int word = lane; word < w / 8; word += 32) {
            uint32_t x = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) x |= (uint32_t)(int)buf[word * 8 + i] << (4 * i);
            reinterpret_cast<uint32_t*>(codes)[word] = x;
        }
    }
    if (lane == 0) {
        pair[0] = scale;
        pair[1] = low;
    }
    __syncwarp();      // buf is free
}

template <typename T, int E, bool kInter, bool kQ4>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a, Geom g, int per_cta, int64_t n_tokens) {
    extern __shared__ __align__(16) float2 cs_all[];         // [per_cta][n_rot / 2]
    __shared__ Token tok[kMaxTokens];
    __shared__ __align__(16) float buf[kQ4 ? kWarps : 1][kQ4 ? kMaxD : 4];
    const int tid = threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.x * per_cta;
    const int n_tok = (int)min((int64_t)per_cta, n_tokens - r0);
    const int half = a.n_rot / 2;
    pdl_wait();
    if (tid < n_tok) {
        const int64_t r = r0 + tid;
        const int b = (int)(r / g.T);
        bool flagged;
        Token t;
        t.row = r;
        t.to = new_row(g, a.kv_rows, r, b, (int)(r - (int64_t)b * g.T), &t.pos, &flagged);
        if (flagged) flag(g.status, IDX_ERR_DEVICE_BOUNDS);
        tok[tid] = t;
    }
    __syncthreads();
    for (int e = tid; e < n_tok * half; e += kThreads) {
        const int i = e / half;
        // (a padding row's queries pass as they are)
        cs_all[e] = tok[i].pos < 0 ? make_float2(1.f, 0.f) : cos_sin(a.inv_freq[e - i * half], tok[i].pos);
    }
    __syncthreads();
    const int uq = head_units<E, kInter>(a, a.dk, true), uv = head_units<E, kInter>(a, a.dv, false);
    const int nq = a.Hq * uq, nk = kQ4 ? 0 : a.Hkv * uq, nv = kQ4 ? 0 : a.Hkv * uv, per = nq + nk + nv;
    // a token's units are shared by the CTAs along y
    const int y0 = (int)((int64_t)per * blockIdx.y / gridDim.y), y1 = (int)((int64_t)per * (blockIdx.y + 1) / gridDim.y);
    const int mine = y1 - y0;
    for (int e = tid; e < n_tok * mine; e += kThreads) {
        const int i = e / mine;
        int u = e - i * mine + y0;
        const Token& t = tok[i];
        const float2* cs = cs_all + i * half;
        const bool is_q = u < nq;
        if (is_q || u < nq + nk) {
            if (!is_q) u -= nq;
            const int h = u / uq;
            u -= h * uq;
            const T* src = is_q ? static_cast<const T*>(a.rows.q) + t.row * a.rows.q_stride : static_cast<const T*>(a.rows.k) + t.row * a.rows.k_stride;
            T* dst = is_q ? static_cast<T*>(a.rows.q_out) + t.row * a.rows.q_out_stride : static_cast<T*>(a.k_cache) + t.to * a.kc_stride;
            if (is_q || t.to >= 0) head_unit<T, E, kInter>(a, src + h * a.dk, dst + h * a.dk, u, a.n_rot > 0, cs);
        } else if (t.to >= 0) {
            u -= nq + nk;       // (the heads of V lie one behind the other: pieces of the whole row)
            store<T, E>(static_cast<T*>(a.v_cache) + t.to * a.vc_stride + u * E,
                        load<T, E>(static_cast<const T*>(a.rows.v) + t.row * a.rows.v_stride + u * E));
        }
    }
    if constexpr (kQ4) {
        const int heads = a.Hkv * (a.rows.v ? 2 : 1);
        const int w0 = (blockIdx.y * kWarps) + (tid >> 5);
        for (int e = w0; e < n_tok * heads; e += kWarps * gridDim.y) {
            const int i = e / heads, hh = e - i * heads;
            const Token& t = tok[i];
            if (t.to < 0) continue;
            const bool is_k = hh < a.Hkv;
            const int h = is_k ? hh : hh - a.Hkv, w = is_k ? a.dk : a.dv;
            const T* src = is_k ? static_cast<const T*>(a.rows.k) + t.row * a.rows.k_stride : static_cast<const T*>(a.rows.v) + t.row * a.rows.v_stride;
            uint8_t* row = is_k ? static_cast<uint8_t*>(a.k_cache) + t.to * a.kc_stride : static_cast<uint8_t*>(a.v_cache) + t.to * a.vc_stride;
            quantize_row<T>(a, src + h * w, w, is_k && a.n_rot > 0, t.pos, cs_all + i * half, buf[tid >> 5], row + h * (w / 2),
                            reinterpret_cast<float*>(row + a.Hkv * (w / 2)) + 2 * h);
        }
    }
}

template <typename T, int E, bool kInter, bool kQ4>
cudaError_t go(const AppendArgs& a, const Geom& g, cudaStream_t st) {
    const int64_t n = (int64_t)g.B * g.T;
    // tokens per CTA: one while there are few, more where a CTA would have little to do
    const int64_t per_tok = ((int64_t)a.Hq * a.dk + (int64_t)a.Hkv * (a.dk + a.dv)) / E;
    int per = 1;
    while (per < kMaxTokens && n / per > 8 * 152 && per_tok * per < 4 * kThreads) per *= 2;
    const int64_t ctas = (n + per - 1) / per;
    // few tokens: several CTAs to one
    int parts = 1;
    while (ctas * parts * 2 <= 152 && per_tok > 2 * kThreads * parts) parts *= 2;
    if (ctas > INT32_MAX) return cudaErrorNotSupported;
    return launch_pdl(append_kernel<T, E, kInter, kQ4>, dim3((unsigned)ctas, (unsigned)parts), dim3(kThreads),
                      sizeof(float2) * per * (a.n_rot / 2), st, a, g, per, n);
}

template <typename T, bool kQ4>
cudaError_t run(const AppendArgs& a, const Geom& g, cudaStream_t st) {
    constexpr int E = 16 / (int)sizeof(T);
    const idx_new_rows& r = a.rows;
    uint64_t all = reinterpret_cast<uintptr_t>(r.q) | reinterpret_cast<uintptr_t>(r.q_out);
    int64_t el = a.n_rot | a.start | (a.interleaved ? 0 : a.n_rot / 2);
    if (r.q) el |= r.q_stride | r.q_out_stride | a.dk;
    if (!kQ4) {
        all |= reinterpret_cast<uintptr_t>(r.k) | reinterpret_cast<uintptr_t>(r.v) | reinterpret_cast<uintptr_t>(a.k_cache) |
               reinterpret_cast<uintptr_t>(a.v_cache);
        el |= r.k_stride | a.kc_stride | a.dk;
        if (r.v) el |= r.v_stride | a.vc_stride | (a.Hkv * a.dv);
        if (r.v && a.dv % E) el |= 1;      // (units count whole pieces of a head)
    }
    const bool vec = all % 16 == 0 && el % E == 0;
    if (a.interleaved) return vec ? go<T, E, true, kQ4>(a, g, st) : go<T, 1, true, kQ4>(a, g, st);
    return vec ? go<T, E, false, kQ4>(a, g, st) : go<T, 1, false, kQ4>(a, g, st);
}

// ------------------------------------------------------------------------------------------- reading back

// a thread per word of eight codes, or per piece of 32 (kWide); kExpand: for the attention (ExpandArgs)
template <typename T, bool kWide, bool kExpand>
__global__ void __launch_bounds__(kThreads) read_q4_kernel(ExpandArgs p, Geom g, int per_cta, int64_t n_rows) {
    __shared__ int64_t at[kThreads];
    constexpr int kCols = kWide ? 32 : 8;
    const ReadArgs& a = p.r;
    const int tid = threadIdx.x;
    pdl_wait();
    const int64_t r0 = (int64_t)blockIdx.x * per_cta;
    const int n = (int)min((int64_t)per_cta, n_rows - r0);
    if (tid < n) {
        const int64_t r = r0 + tid;
        const int b = (int)(r / g.T), t = (int)(r - (int64_t)b * g.T);
        int64_t row = -1;
        if (kExpand) {
            const int2 span = p.span[b];
            if (t >= span.x && t < span.y) {
                row = key_row(g, b, t);
                if (row < 0 || row >= a.kv_rows) {
                    *p.lost = 1;
                    row = -1;
                }
            }
        } else {
            int pos;
            bool flagged;
            row = new_row(g, a.kv_rows, r, b, t, &pos, &flagged);
            if (flagged) flag(g.status, IDX_ERR_DEVICE_BOUNDS);
        }
        at[tid] = row;
    }
    __syncthreads();
    const int pk = a.Hkv * (a.dk / kCols), pv = a.Hkv * (a.dv / kCols), per = pk + pv;
    for (int e = tid; e < n * per; e += kThreads) {
        const int i = e / per;
        int u = e - i * per;
        const int64_t row = at[i];
        if (row < 0) continue;
        const bool is_k = u < pk;
        if (!is_k) u -= pk;
        const int w = is_k ? a.dk : a.dv, ph = w / kCols, h = u / ph;
        const uint8_t* src = is_k ? static_cast<const uint8_t*>(a.k_cache) + row * a.kc_stride
                                  : static_cast<const uint8_t*>(a.v_cache) + row * a.vc_stride;
        T* dst = (is_k ? static_cast<T*>(a.k_out) : static_cast<T*>(a.v_out)) + ((r0 + i) * a.Hkv * w + u * kCols);
        T* rest = kExpand ? static_cast<T*>(p.k_rest) + (dst - static_cast<T*>(a.k_out)) : nullptr;
        const float* pair = reinterpret_cast<const float*>(src + a.Hkv * (w / 2)) + 2 * h;
        const float scale = pair[0], low = pair[1];
        uint32_t x[kCols / 8];
        if constexpr (kWide)
            *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(src + u * 16);
        else
            x[0] = *reinterpret_cast<const uint32_t*>(src + u * 4);
        constexpr int E = 16 / (int)sizeof(T);
#pragma unroll
        for (int c = 0; c < kCols; c += E) {
            T y[E], z[E];
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float v = fmaf((float)((x[(c + j) / 8] >> (4 * ((c + j) % 8))) & 15u), scale, low);
                y[j] = from_f32<T>(v);
                if (kExpand) z[j] = from_f32<T>(v - to_f32(y[j]));
            }
            if (kExpand && is_k) *reinterpret_cast<uint4*>(rest + c) = *reinterpret_cast<const uint4*>(z);
            *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(y);
        }
    }
}

template <typename T, bool kExpand>
cudaError_t run_read(const ExpandArgs& p, const Geom& g, cudaStream_t st) {
    const ReadArgs& a = p.r;
    const int64_t n = (int64_t)g.B * g.T;
    const uint64_t all = reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache) | (uint64_t)a.kc_stride |
                         (a.v_cache ? (uint64_t)a.vc_stride : 0) | (uint64_t)(a.dk / 2) | (uint64_t)(a.dv / 2);
    const bool wide = all % 16 == 0;
    const int64_t per_row = (int64_t)a.Hkv * (a.dk + a.dv) / (wide ? 32 : 8);
    int per = 1;
    while (per < kThreads && per_row * per < 2 * kThreads && n / per > 2 * 152) per *= 2;
    const int64_t ctas = (n + per - 1) / per;
    if (ctas > INT32_MAX) return cudaErrorNotSupported;
    return wide ? launch_pdl(read_q4_kernel<T, true, kExpand>, dim3((unsigned)ctas), dim3(kThreads), 0, st, p, g, per, n)
                : launch_pdl(read_q4_kernel<T, false, kExpand>, dim3((unsigned)ctas), dim3(kThreads), 0, st, p, g, per, n);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int dtype, bool q4, const Geom& g, cudaStream_t st) {
    switch (dtype) {
        case IDX_F16: return q4 ? run<__half, true>(a, g, st) : run<__half, false>(a, g, st);
        case IDX_BF16: return q4 ? run<__nv_bfloat16, true>(a, g, st) : run<__nv_bfloat16, false>(a, g, st);
        default: return q4 ? run<float, true>(a, g, st) : run<float, false>(a, g, st);
    }
}

cudaError_t launch_read_q4(const ReadArgs& a, int dtype, const Geom& g, cudaStream_t st) {
    ExpandArgs p = {};
    p.r = a;
    switch (dtype) {
        case IDX_F16: return run_read<__half, false>(p, g, st);
        case IDX_BF16: return run_read<__nv_bfloat16, false>(p, g, st);
        default: return run_read<float, false>(p, g, st);
    }
}

cudaError_t launch_expand_q4(const ExpandArgs& a, int dtype, const Geom& g, cudaStream_t st) {
    return dtype == IDX_BF16 ? run_read<__nv_bfloat16, true>(a, g, st) : run_read<__half, true>(a, g, st);
}

}  // namespace lidx
