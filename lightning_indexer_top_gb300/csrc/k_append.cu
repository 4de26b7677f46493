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
// alignments go element by element.  A chunk of 4096 bf16 tokens with 32 + 4 + 4 heads of
// 128, 84 MB: 18 us = 4.6 TB/s; it waits for its loads, which six CTAs to an SM hide best.  The
// rows of one decode step of 16 sequences: 3 us, which is the launch and four loads one
// after another.
//
// 4 bits: the codes of a head row are made in registers by a power of two of lanes, sixteen
// columns to a lane, from f32 while f32 can tell the codes apart.  8192 bf16 tokens with
// 32 + 8 + 8 heads of 128, 201 MB: 74 us = 2.7 TB/s; loads are waited for and issue slots are
// two fifths used, four CTAs to an SM at 64 registers (three or five: 77 us).
#include <float.h>

#include <algorithm>

#include "q4.cuh"

namespace lidx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 16;     // per CTA
constexpr int kMaxCs = 2048;       // pairs of cosine and sine per CTA
constexpr int kMaxD = 576;

// Phase of position p in turns of 2^64: the fraction of f / 2 pi, times p.  In whole numbers: f = m 2^e with |m| < 2^24, and
// 1 / 2 pi to 96 bits, good to 2^-63 of a turn for |f| < 2^24 (64-bit floats, which are scarce here, beyond).  Cut off at 2^-64 of
// a turn whatever f, so the phase is good to p times that, not to a part of p f.
__device__ __forceinline__ uint64_t phase(float f, int p) {
    const uint32_t bits = __float_as_uint(f);
    const int e = max((int)(bits >> 23 & 255u), 1) - 150;            // f = m 2^e
    const uint64_t m = (bits & 0x7fffffu) | (bits & 0x7f800000u ? 0x800000u : 0u);
    uint64_t u;
    if (e <= 0) {
        // m * (2^96 / 2 pi): bits 0 .. 63 and 64 .. 127
        const uint64_t p0 = m * 0x7f09d5f4u, p1 = m * 0x9391054au + (p0 >> 32), p2 = m * 0x28be60dbu + (p1 >> 32);
        const uint64_t low = p1 << 32 | (uint32_t)p0;
        const int s = 32 - e;                                        // the fraction's top 64 bits: from bit s on
        u = s < 64 ? (s ? p2 << (64 - s) : 0) | low >> s : s < 128 ? p2 >> (s - 64) : 0;
        if (bits >> 31) u = 0 - u;
    } else {
        const double turns = (double)f * 0.15915494309189533577;     // 1 / 2 pi
        u = (uint64_t)((turns - floor(turns)) * 18446744073709551616.0);     // (a fraction of 1 saturates)
    }
    return u * (uint64_t)(uint32_t)p;
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

// A thread's piece of work: one piece of E columns, or two that are turned together.
template <typename T>
struct Unit {
    const T* src;          // NULL: nothing
    T* dst;
    const float2* cs;      // NULL: as it is
    int apart;             // the second piece, 0: none
};

// Unit u of a head row of w columns (rot: rotated): with the pairs apart, first the n_rot / 2 / E pairs of pieces, then the
// columns that stay; with the pairs side by side, pieces of E columns.
template <typename T, int E, bool kInter>
__device__ __forceinline__ Unit<T> head_unit(const AppendArgs& a, const T* src, T* dst, int u, bool rot, const float2* cs) {
    const int n = rot ? a.n_rot : 0;
    int c;
    Unit<T> x = {src, dst, nullptr, 0};
    if (kInter && E > 1) {
        c = u * E;
        if (c >= a.start && c < a.start + n) x.cs = cs + (c - a.start) / 2;
    } else if (u < n / (2 * E)) {
        c = kInter ? a.start + 2 * u : a.start + u * E;
        x.cs = cs + u * E;
        x.apart = kInter ? 1 : n / 2;
    } else {
        c = (u - n / (2 * E)) * E;
        if (c >= a.start) c += n;
    }
    x.src += c;
    x.dst += c;
    return x;
}

template <typename T, int E, bool kInter>
__device__ __forceinline__ void finish(const Unit<T>& x, Piece<T, E>& v, Piece<T, E>& w) {
    if (x.cs) {
        if (kInter && E > 1) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 t = x.cs[i];
                const float y = to_f32(v.x[2 * i]), z = to_f32(v.x[2 * i + 1]);
                v.x[2 * i] = from_f32<T>(fmaf(y, t.x, -(z * t.y)));
                v.x[2 * i + 1] = from_f32<T>(fmaf(z, t.x, y * t.y));
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float2 t = x.cs[i];
                const float y = to_f32(v.x[i]), z = to_f32(w.x[i]);
                v.x[i] = from_f32<T>(fmaf(y, t.x, -(z * t.y)));
                w.x[i] = from_f32<T>(fmaf(z, t.x, y * t.y));
            }
            store<T, E>(x.dst + x.apart, w);
        }
    }
    store<T, E>(x.dst, v);
}

// units of a head row of w columns
template <int E, bool kInter>
__device__ __forceinline__ int head_units(const AppendArgs& a, int w, bool rot) {
    return kInter && E > 1 ? w / E : rot ? (w - a.n_rot / 2) / E : w / E;
}

// ------------------------------------------------------------------------------------------- 4 bits

// column c of a head row after the rotation in 64 bits
template <typename T>
__device__ __noinline__ double exact_column(const AppendArgs& a, const T* src, int c, bool rot, int p) {
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

// A warp's head row of w columns into 4 bits at `codes` and `pair`, in 64 bits (buf: w floats of shared memory).
template <typename T>
__device__ __noinline__ void exact_row(const AppendArgs& a, const T* src, int w, bool rot, int p, float* buf, uint8_t* codes, float* pair) {
    const int lane = threadIdx.x & 31;
    double lo = INFINITY, hi = -INFINITY;
    bool fine = true;
    for (int c = lane; c < w; c += 32) {
        fine &= fabsf(to_f32(src[c])) <= FLT_MAX;
        const double y = exact_column(a, src, c, rot, p);
        lo = fmin(lo, y);
        hi = fmax(hi, y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    fine = __all_sync(0xffffffffu, fine);
    const double span = hi - lo;
    for (int c = lane; c < w; c += 32)
        buf[c] = fine && span > 0.0 ? (float)rint((exact_column(a, src, c, rot, p) - lo) * 15.0 / span) : 0.f;
    __syncwarp();
    for (int word = lane; word < w / 8; word += 32) {
        uint32_t x = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) x |= (uint32_t)(int)buf[word * 8 + i] << (4 * i);
        reinterpret_cast<uint32_t*>(codes)[word] = x;
    }
    if (lane == 0) {
        pair[0] = fine ? (float)(span / 15.0) : __int_as_float(0x7fc00000);
        pair[1] = fine ? (float)lo : __int_as_float(0x7fc00000);
    }
    __syncwarp();      // buf is free
}

// Codes from f32.  Rotated, a column is off by at most 1.25 * 2^-22 of its pair's |u| + |w| (the angle by pi * 2^-25, cosine and
// sine by an ulp, three roundings), so t = 15 (x - min) / (max - min) by at most 60 such errors over max - min, and
// 15 * 2^-22 for its own roundings.  A row with a column that lies nearer than that to a border between codes is done again in
// 64 bits (one head row of 128 in about 200), and so is one whose span, or its inverse, is no number above 0.
struct Scale {
    float lo, span, inv, eps;
    bool sure;
    __device__ __forceinline__ Scale(float low, float high, float big) {
        lo = low;
        span = high - low;
        inv = 15.f / span;
        eps = (60.f * 1.25f * 0x1p-22f) * big / span + 15.f * 0x1p-22f;
        sure = inv <= FLT_MAX && inv > 0.f && span <= FLT_MAX && eps < 0.25f;
    }
    // The code of y, in the low bits of kRound's (kRound + code is the nearest whole number to t); near: f32 does not tell
    static constexpr float kRound = 12582912.f;                 // 1.5 * 2^23
    static constexpr uint32_t kRoundBits = 0x4B400000u;
    __device__ __forceinline__ uint32_t code(float y, bool& near) const {
        const float d = y - lo, r = fmaf(d, inv, kRound);
        near = !(fabsf(fmaf(d, inv, kRound - r)) <= 0.5f - eps);
        return __float_as_uint(r);
    }
    // The code of a column near a border where columns are exact (not rotated): the sign of 15 (y - lo) - (k + 1/2) (hi - lo), in
    // f32 where both differences are f32s.  Values on a coarse grid, as 16-bit ones are, meet borders often: a quarter of the
    // rows of 128 bf16 columns have one that lies on a border exactly.
    __device__ __forceinline__ int border(float y, float high, bool& near) const {
        auto rest = [](float x, float z, float d) {       // of d = x - z rounded: 0 where it is exact
            const float v = d - x;
            return (x - (d - v)) - (z + v);
        };
        const float d = y - lo, k = floorf(d * inv), p = 15.f * d, e = fmaf(15.f, d, -p), q = fmaf(k + 0.5f, span, -p);
        near = rest(y, lo, d) != 0.f || rest(high, lo, span) != 0.f || !(e == 0.f || fabsf(q) > 2.f * fabsf(e));
        return (int)k + (q < 0.f || (q == 0.f && ((int)k & 1)) ? 1 : 0);
    }
};

// a warp's head row, of any width, start and alignment
template <typename T>
__device__ __forceinline__ void quantize_row(const AppendArgs& a, const T* src, int w, bool rot, int p, const float2* cs,
                                             float* buf, uint8_t* codes, float* pair) {
    const int lane = threadIdx.x & 31;
    const int n = rot ? a.n_rot : 0, half = n / 2;
    float big = 0.f;       // the largest |u| + |w|
    float lo = INFINITY, hi = -INFINITY;
    auto take = [&](int c, float y) {
        buf[c] = y;
        lo = fminf(lo, y);
        hi = fmaxf(hi, y);
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
    __syncwarp();
    const Scale s(lo, hi, big);
    bool near = !s.sure;       // (a NaN is near any border)
    for (int word = lane; word < w / 8; word += 32) {
        const float4 y0 = *reinterpret_cast<const float4*>(buf + word * 8), y1 = *reinterpret_cast<const float4*>(buf + word * 8 + 4);
        const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
        uint32_t x = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bool n8;
            x |= (s.code(y[i], n8) & 15u) << (4 * i);
            near |= n8;
        }
        if (!near) reinterpret_cast<uint32_t*>(codes)[word] = x;
    }
    if (__any_sync(0xffffffffu, near)) {
        exact_row(a, src, w, rot, p, buf, codes, pair);
        return;
    }
    if (lane == 0) {
        pair[0] = s.span / 15.f;
        pair[1] = lo;
    }
    __syncwarp();      // buf is free
}

// eight columns at p
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; i += 16 / (int)sizeof(T)) *reinterpret_cast<uint4*>(v + i) = *reinterpret_cast<const uint4*>(p + i);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(v[i]);
}

// the larger one, a NaN where either is one
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// Head rows whose columns come in aligned eights: a lane has two of those, the ones that are turned together or neighbours, and
// `lanes` (a power of two, at least w / 16) of them a row.  src NULL: no row for this lane.  False: the row is to be done in
// 64 bits, as is one that holds a NaN or an infinity: a NaN passes through the maximum, an infinity leaves no span.
template <typename T>
__device__ __forceinline__ bool quantize_group(const AppendArgs& a, const T* src, int w, int lanes, bool rot, int p, const float2* cs,
                                               uint8_t* codes, float* pair) {
    const int li = threadIdx.x & (lanes - 1);
    const int n = rot ? a.n_rot : 0;
    const bool on = src && li < w / 16;
    float x[2][8], big = 0.f, lo = INFINITY, hi = -INFINITY;
    int c[2] = {16 * li, 16 * li + 8};
    if (n && !a.interleaved) {
        if (li < n / 16) {
            c[0] = a.start + 8 * li;
            c[1] = c[0] + n / 2;
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                c[e] -= n;
                if (c[e] >= a.start) c[e] += n;
            }
        }
    }
    if (on) {
        load8(src + c[0], x[0]);
        load8(src + c[1], x[1]);
        if (n && a.interleaved) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (c[e] < a.start || c[e] >= a.start + n) continue;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 t = cs[(c[e] - a.start + i) / 2];
                    const float u = x[e][i], v = x[e][i + 1];
                    big = fmaxf(big, fabsf(u) + fabsf(v));
                    x[e][i] = fmaf(u, t.x, -(v * t.y));
                    x[e][i + 1] = fmaf(v, t.x, u * t.y);
                }
            }
        } else if (li < n / 16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 t = cs[8 * li + i];
                const float u = x[0][i], v = x[1][i];
                big = fmaxf(big, fabsf(u) + fabsf(v));
                x[0][i] = fmaf(u, t.x, -(v * t.y));
                x[1][i] = fmaf(v, t.x, u * t.y);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo = fminf(lo, x[e][i]);
                hi = max_nan(hi, x[e][i]);
            }
    }
    for (int o = lanes >> 1; o; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    }
    const uint32_t mine = lanes == 32 ? ~0u : ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
    const Scale s(lo, hi, big);
    float scale = s.span / 15.f, low = lo;
    uint32_t word[2] = {0u, 0u};
    bool any = false;          // a column that f32 does not tell
    bool other = false;        // neither a span to divide by nor the same number throughout (whose codes are 0)
    if (on && !s.sure) {
        other = big > 0.f || !(fabsf(lo) <= FLT_MAX);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 8; ++i) other |= !(x[e][i] == lo);
    } else if (on) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                bool near;
                word[e] += s.code(x[e][i], near) << (4 * i);
                any |= near;
            }
            word[e] -= 0x11111111u * Scale::kRoundBits;
        }
    }
    const bool sure = !(__ballot_sync(0xffffffffu, other) & mine);
    if (__any_sync(0xffffffffu, any)) {
        // (one place for each kind of work: bit 8 e + i for column c[e] + i)
        uint64_t w = (uint64_t)word[1] << 32 | word[0];
        auto put = [&](int at, int k) { w = (w & ~(15ull << (4 * at))) | (uint64_t)k << (4 * at); };
        auto column = [&](int at) { return (at < 8 ? c[0] : c[1]) + (at & 7); };
        uint32_t nears = 0u;
        if (any) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    bool near;
                    s.code(x[e][i], near);
                    nears |= near ? 1u << (8 * e + i) : 0u;
                }
            if (big == 0.f)
                for (uint32_t left = nears; left; left &= left - 1) {
                    const int at = __ffs(left) - 1;
                    bool near;
                    put(at, s.border(to_f32(src[column(at)]), hi, near));
                    if (!near) nears &= ~(1u << at);
                }
        }
        __syncwarp();
        const bool hit = __ballot_sync(0xffffffffu, nears) & mine;
        if (__any_sync(0xffffffffu, hit)) {
            // In 64 bits: the columns that may be the row's least and largest, and those near a border (a row of 128 rotated
            // columns has one in 200 times).
            const float err = 2.f * 1.25f * 0x1p-22f * big;
            double least = INFINITY, most = -INFINITY;
            uint32_t low_at = 0u, high_at = 0u;
            if (hit && on) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        low_at |= x[e][i] <= lo + err ? 1u << (8 * e + i) : 0u;
                        high_at |= x[e][i] >= hi - err ? 1u << (8 * e + i) : 0u;
                    }
            }
            for (uint32_t left = low_at | high_at; left; left &= left - 1) {
                const int at = __ffs(left) - 1;
                const double y = exact_column(a, src, column(at), rot, p);
                if ((low_at >> at) & 1u) least = fmin(least, y);
                if ((high_at >> at) & 1u) most = fmax(most, y);
            }
            __syncwarp();
            for (int o = lanes >> 1; o; o >>= 1) {
                least = fmin(least, __shfl_xor_sync(0xffffffffu, least, o));
                most = fmax(most, __shfl_xor_sync(0xffffffffu, most, o));
            }
            if (hit) {
                scale = (float)((most - least) / 15.0);
                low = (float)least;
            }
            for (uint32_t left = nears; left; left &= left - 1) {
                const int at = __ffs(left) - 1;
                const double t = rint((exact_column(a, src, column(at), rot, p) - least) * 15.0 / (most - least));
                put(at, (int)fmin(fmax(t, 0.0), 15.0));
            }
            __syncwarp();
        }
        word[0] = (uint32_t)w;
        word[1] = (uint32_t)(w >> 32);
    }
    if (on && sure) {
        reinterpret_cast<uint32_t*>(codes)[c[0] / 8] = word[0];
        reinterpret_cast<uint32_t*>(codes)[c[1] / 8] = word[1];
        if (li == 0) {
            pair[0] = scale;
            pair[1] = low;
        }
    }
    return sure || !src;
}

template <typename T, int E, bool kInter, bool kQ4>
__global__ void __launch_bounds__(kThreads, kQ4 ? 4 : 6) append_kernel(AppendArgs a, Geom g, int per_cta, int64_t n_tokens) {
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
    auto unit = [&](int e) -> Unit<T> {
        const int i = e / mine;
        int u = e - i * mine + y0;
        const Token& t = tok[i];
        if (u < nq) {
            const int h = u / uq;
            return head_unit<T, E, kInter>(a, static_cast<const T*>(a.rows.q) + t.row * a.rows.q_stride + h * a.dk,
                                           static_cast<T*>(a.rows.q_out) + t.row * a.rows.q_out_stride + h * a.dk, u - h * uq, a.n_rot > 0,
                                           cs_all + i * half);
        }
        if (t.to < 0) return {nullptr, nullptr, nullptr, 0};
        u -= nq;
        if (u < nk) {
            const int h = u / uq;
            return head_unit<T, E, kInter>(a, static_cast<const T*>(a.rows.k) + t.row * a.rows.k_stride + h * a.dk,
                                           static_cast<T*>(a.k_cache) + t.to * a.kc_stride + h * a.dk, u - h * uq, a.n_rot > 0,
                                           cs_all + i * half);
        }
        u -= nk;       // (the heads of V lie one behind the other: pieces of the whole row)
        return {static_cast<const T*>(a.rows.v) + t.row * a.rows.v_stride + u * E,
                static_cast<T*>(a.v_cache) + t.to * a.vc_stride + u * E, nullptr, 0};
    };
    // (two or three units' loads at a time: 30 and 42 us for 18 of a 4096-token bf16 chunk, 34 and 39 for 31 in f32, 7.7 and 8.4 for
    // 7.2 of 8192 latent rows)
    for (int e = tid; e < n_tok * mine; e += kThreads) {
        const Unit<T> x = unit(e);
        if (!x.src) continue;
        Piece<T, E> v = load<T, E>(x.src), w;
        if (x.apart) w = load<T, E>(x.src + x.apart);
        finish<T, E, kInter>(x, v, w);
    }
    if constexpr (kQ4) {
        const int warp = tid >> 5, lane = tid & 31;
        for (int kind = 0; kind < (a.rows.v ? 2 : 1); ++kind) {
            const bool is_k = kind == 0, rot = is_k && a.n_rot > 0;
            const int w = is_k ? a.dk : a.dv, rows = n_tok * a.Hkv;
            struct Row {
                const T* src;
                uint8_t* codes;
                float* pair;
                int i;
            };
            auto row_at = [&](int e) -> Row {
                Row r = {nullptr, nullptr, nullptr, e / a.Hkv};
                if (e >= rows || tok[r.i].to < 0) return r;
                const int h = e - r.i * a.Hkv;
                const Token& t = tok[r.i];
                uint8_t* c = is_k ? static_cast<uint8_t*>(a.k_cache) + t.to * a.kc_stride
                                  : static_cast<uint8_t*>(a.v_cache) + t.to * a.vc_stride;
                r.src = (is_k ? static_cast<const T*>(a.rows.k) + t.row * a.rows.k_stride
                              : static_cast<const T*>(a.rows.v) + t.row * a.rows.v_stride) + h * w;
                r.codes = c + h * (w / 2);
                r.pair = reinterpret_cast<float*>(c + a.Hkv * (w / 2)) + 2 * h;
                return r;
            };
            int lanes = is_k ? a.k_lanes : a.v_lanes;
            if (lanes) {
                const int per = 32 / lanes;
                for (int e = (blockIdx.y * kWarps + warp) * per; e < rows; e += kWarps * gridDim.y * per) {
                    const Row r = row_at(e + lane / lanes);
                    const int tk = min(r.i, n_tok - 1);
                    const bool done = quantize_group(a, r.src, w, lanes, rot, tok[tk].pos, cs_all + tk * half, r.codes, r.pair);
                    // (a lane of each row that is not)
                    uint32_t left = __ballot_sync(0xffffffffu, !done && (lane & (lanes - 1)) == 0);
                    for (; left; left &= left - 1) {
                        const Row x = row_at(e + (__ffs(left) - 1) / lanes);
                        exact_row(a, x.src, w, rot, tok[x.i].pos, buf[warp], x.codes, x.pair);
                    }
                }
            } else {
                for (int e = blockIdx.y * kWarps + warp; e < rows; e += kWarps * gridDim.y) {
                    const Row r = row_at(e);
                    if (r.src) quantize_row(a, r.src, w, rot, tok[r.i].pos, cs_all + r.i * half, buf[warp], r.codes, r.pair);
                }
            }
        }
    }
}

template <typename T, int E, bool kInter, bool kQ4>
cudaError_t go(const AppendArgs& a, const Geom& g, cudaStream_t st) {
    const int64_t n = (int64_t)g.B * g.T;
    // Tokens per CTA: one while there are few, then what makes a round of CTAs (two rounds with 4 bits), the last one not
    // over: a token's first loads (lengths, positions, pages) and its cosines take longer than its rows.  Rounded down
    // instead: 8192 4-bit tokens 76 us for 74, 2048 of them 32 for 27, 8192 16-bit tokens 36 for 32.
    const int64_t per_tok = ((int64_t)a.Hq * a.dk + (int64_t)a.Hkv * (a.dk + a.dv)) / E;
    constexpr int kAll = 152 * (kQ4 ? 8 : 6);
    int per = (int)std::min<int64_t>((n + kAll - 1) / kAll, kMaxTokens);
    if (per * a.n_rot > kMaxCs * 2) per = kMaxCs * 2 / a.n_rot;
    if (per < 1) per = 1;
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
    AppendArgs b = a;
    if (kQ4) {
        // lanes of a head row whose columns come in aligned eights, up to a warp
        auto lanes = [&](const void* x, int64_t stride, int w, bool rot) {
            if (!x || reinterpret_cast<uintptr_t>(x) % 16 || stride * (int64_t)sizeof(T) % 16 || w * (int64_t)sizeof(T) % 16 ||
                w % 16 || w > 512)
                return 0;
            if (rot && (a.start % 8 || a.n_rot % (a.interleaved ? 8 : 16))) return 0;
            int n = 1;
            while (n < w / 16) n *= 2;
            return n;
        };
        b.k_lanes = lanes(r.k, r.k_stride, a.dk, a.n_rot > 0);
        b.v_lanes = lanes(r.v, r.v_stride, a.dv, false);
    }
    if (a.interleaved) return vec ? go<T, E, true, kQ4>(b, g, st) : go<T, 1, true, kQ4>(b, g, st);
    return vec ? go<T, E, false, kQ4>(b, g, st) : go<T, 1, false, kQ4>(b, g, st);
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
        const float k_unit = kExpand && is_k && p.k_top ? exp2_whole(-k_exponent(p.k_top[(r0 + i) / g.T * a.Hkv + h])) : 1.f;
        if (kExpand && is_k && isfinite(scale) && isfinite(low)) {
            // (numbers, but not of type T; or with a power of two below what two parts have 22 bits for)
            const float most = fmaxf(fabsf(low), fabsf(fmaf(15.f, scale, low))) * k_unit;
            if (isinf(to_f32(from_f32<T>(most))) || (p.k_top && most > 0.f && most < 0x1p-3f)) *p.lost = 1;
        }
        uint32_t x[kCols / 8];
        if constexpr (kWide)
            *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(src + u * 16);
        else
            x[0] = *reinterpret_cast<const uint32_t*>(src + u * 4);
        constexpr int E = 16 / (int)sizeof(T);
        if (kExpand && !is_k) {
            const float f = exp2_whole(-v_exponent(p.v_top[(r0 + i) / g.T * a.Hkv + h]));
            // (of a key far below the largest f16 would keep fewer bits, or none: rows that do not see the largest need them)
            const float most = fmaxf(fabsf(low), fabsf(fmaf(15.f, scale, low)));
            if (isfinite(scale) && isfinite(low) && most > 0.f && most * f < 0x1p-14f) *p.lost = 1;
#pragma unroll
            for (int c = 0; c < kCols; c += 8) {
                __half y[8], z[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = fmaf((float)((x[c / 8] >> (4 * j)) & 15u), scale, low) * f;
                    y[j] = from_f32<__half>(v);
                    z[j] = from_f32<__half>(v - to_f32(y[j]));
                }
                *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(y);
                T* v_rest = static_cast<T*>(p.v_rest);
                if (v_rest) *reinterpret_cast<uint4*>(v_rest + (dst - static_cast<T*>(a.v_out)) + c) = *reinterpret_cast<const uint4*>(z);
            }
            continue;
        }
#pragma unroll
        for (int c = 0; c < kCols; c += E) {
            T y[E], z[E];
#pragma unroll
            for (int j = 0; j < E; ++j) {
                float v = fmaf((float)((x[(c + j) / 8] >> (4 * ((c + j) % 8))) & 15u), scale, low);
                if (kExpand) v *= k_unit;
                y[j] = from_f32<T>(v);
                if (kExpand) z[j] = from_f32<T>(v - to_f32(y[j]));
            }
            if (kExpand) *reinterpret_cast<uint4*>(rest + c) = *reinterpret_cast<const uint4*>(z);
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
