// Dense attention over 4-bit caches (dense_attn_q4 in lidx.h): few rows, and the choice of the way.
//
// Few rows (16-bit q, heads of 64 or 128): a warp multiplies the codes themselves, expanded in registers to the operands of
// mma.sync, so that nothing but the packed bytes moves.  With code n, scale s, minimum m and m' = m + 8 s a value is
// s (n - 8) + m', and n - 8 is exact in f16 and bf16:
//     scores  x[j] = s_j (q . (n_j - 8)) + m'_j sum(q)               keys are the M side, rows (tokens x heads) the N side
//     output  O    = sum_j (p_j s_j) (n_j - 8) + sum_j p_j m'_j      columns are the M side, rows the N side
// q is brought to f16 at a power of two of its row's (exact but for what lies 2^-27 below the row's largest), and the
// weights p_j s_j are rounded to f16 at a running maximum of theirs; centring the codes keeps that rounding as small as
// the values' own.  For bf16 results that is little beside their own rounding (0.0017 of the result with and without); f16
// results would be off by 1.3 times theirs, so there what the weights lack is a second operand (the decode below, in f16: 70 us
// for 67).  The order of columns within a product is free, so a lane takes 16 bytes of a key's codes as they lie and q
// is laid out to match.
//
// 16 sequences of up to 32768 keys, 32 bf16 heads of 128 on 4, 64-row pages: 67 us for 231 MB, 3.4 TB/s.  Not memory bounds it
// but the way from codes to operands: schedulers issue on half of the cycles, three warps to each, mostly waiting for their own
// last result (tensor pipe 20 %, ALU 49 %).  No better: four CTAs to an SM at 128 registers, two to five blocks ahead, halves
// of a block one after the other (66 to 68), V expanded before the softmax (69), eight warps to a CTA (79), scales by plain
// copies instead of TMA's (66 to 69).
#include <algorithm>

#include "q4.cuh"
#include "sm100_ptx.cuh"

namespace lidx {
namespace {
using namespace sm100;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlock = 32;                   // keys a warp works on at a time, in two halves
constexpr int kTile = 128;                   // keys by which a row's are cut
// Packed rows up to which the codes themselves are multiplied, 16 to a tile, each tile expanding them anew.  With the expanded
// K and V: 16 x 128 rows on up to 32768 keys 841 us, this way 499; 16 x 256 897 and 785; 1 x 512 132 and 206.
constexpr int kManyRows = 256;
constexpr float kShift = 7.f, kTop = kShift + 8.f;
constexpr int kMinTiles = 2;                 // a piece of a row's keys, at least

struct Q4Args {
    DenseArgs a;
    int row_tiles;       // tiles of 8 NB packed rows per (sequence, kv head)
    int slots;           // CTAs wanted; 0: a row's keys are one piece
    int box;             // rows of a TMA box: the largest power of two that divides the page, at most kBlock; 0: below 8
    int shift;           // log2 of the page size, -1: of another one
    uint32_t pages;      // pages that hold a row of the cache
    float* part_o;       // [CTA][8 NB][D] unnormalised
    float* part_ml;      // [CTA][8 NB][2]: maximum (log2 units), sum
};

struct Maps {
    CUtensorMap k, v, k_pair, v_pair;
};

// Pieces: a row's keys are cut so that the pieces of all rows are about as long, and few enough to run at once.  est: tiles
// that a sequence's rows are taken to see (masks aside; it only shapes the cuts).
struct Cut {
    int b, piece, pieces;      // b < 0: nothing
    int first;                 // index of the sequence's first piece
};

__device__ __forceinline__ int est_tiles(const Geom& g, const idx_attn_mods& m, int b) {
    int n = g.n_kv[b];
    n = min(max(n, 0), g.max_n_kv);
    if (m.window > 0 && !m.prefix_len && !m.prefix_end && (int64_t)m.window + g.T < n) n = m.window + g.T;
    return (n + kTile - 1) / kTile;
}

// every lane of a warp comes here; by_piece: the piece `at` of the line of all pieces, else those of sequence `at`
__device__ __forceinline__ Cut cut_of(const Geom& g, const Q4Args& p, int at, bool by_piece) {
    const int lane = threadIdx.x & 31;
    Cut c = {-1, 0, 1, 0};
    if (!p.slots) {
        if (at < g.B) c = {at, 0, 1, at};
        return c;
    }
    const int64_t columns = (int64_t)p.a.Hkv * p.row_tiles;
    const int few = lane < g.B ? est_tiles(g, p.a.mods, lane) : 0;      // (the first 32 sequences' stay at hand)
    auto est = [&](int b0) { return b0 == 0 ? few : b0 + lane < g.B ? est_tiles(g, p.a.mods, b0 + lane) : 0; };
    int64_t total = 0;
    for (int b0 = 0; b0 < g.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, est(b0));
    int len = (int)min((total * columns + p.slots - 1) / p.slots, (int64_t)1 << 25);
    if (len < kMinTiles) len = kMinTiles;
    auto pieces_of = [&](int b0) { return b0 + lane < g.B ? max((est(b0) + len - 1) / len, 1) : 0; };
    // (rounding up each row's pieces takes more than the slots: longer ones, a few tries)
    for (int i = 0; i < 4; ++i) {
        int64_t n = 0;
        for (int b0 = 0; b0 < g.B; b0 += 32) n += __reduce_add_sync(0xffffffffu, pieces_of(b0));
        if (n * columns <= p.slots) break;
        len += (len + 15) / 16;
    }
    int before = 0;
    for (int b0 = 0; b0 < g.B; b0 += 32) {
        const int mine = pieces_of(b0);
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const int first = before + incl - mine;
        const bool hit = b0 + lane < g.B && (by_piece ? at >= first && at < first + mine : at == b0 + lane);
        const uint32_t who = __ballot_sync(0xffffffffu, hit);
        if (who) {
            const int src = __ffs(who) - 1;
            c.b = b0 + src;
            c.first = __shfl_sync(0xffffffffu, first, src);
            c.pieces = __shfl_sync(0xffffffffu, mine, src);
            c.piece = by_piece ? at - c.first : 0;
            return c;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return c;
}

__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
    return r;
}
__device__ __forceinline__ uint32_t h2(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// codes i (0 .. 3) of a word's two halves as a pair of f16: n - 8.  A code under the exponent of 1024 is the f16 1024 + n, or
// 1024 + 16 n, from which one addition or FMA takes the rest (Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't Run", 2022).
// kRaw: the odd ones stay 1024 + 16 n = 16 (n - 8 + 72), and
// the product's user takes 72 (and 16) off again: two instructions less, for K's sums of D terms.  (V's run over all keys: with
// 72 too much in them their f32 rounding showed, an error of 0.4 % on averages over 30000 keys.)
template <bool kRaw>
__device__ __forceinline__ void codes(uint32_t w, uint32_t (&o)[4]) {
    const __half2 c = __float2half2_rn(-1032.f);
    const uint32_t v = w >> 8;
    o[0] = h2(__hadd2(as_h2(and_or(w, 0x000f000fu, 0x64006400u)), c));       // 1024 + n
    o[1] = and_or(w, 0x00f000f0u, 0x64006400u);
    o[2] = h2(__hadd2(as_h2(and_or(v, 0x000f000fu, 0x64006400u)), c));
    o[3] = and_or(v, 0x00f000f0u, 0x64006400u);
    if (!kRaw) {
        o[1] = h2(__hfma2(as_h2(o[1]), __float2half2_rn(0.0625f), __float2half2_rn(-72.f)));
        o[3] = h2(__hfma2(as_h2(o[3]), __float2half2_rn(0.0625f), __float2half2_rn(-72.f)));
    }
}
constexpr float kOdd = 72.f;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a b + (c0, c1, c0, c1)
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, float c0,
                                         float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A block in a warp's ring in shared memory, brought by TMA in boxes of at least eight rows (a box starts on 128 bytes): rows
// of 64 bytes in the 64-byte swizzle (the 16-byte pieces of row r at r / 2 % 4 ^ piece), shorter ones as they lie; scale and
// minimum of two neighbouring heads.  Pages that are no multiple of eight rows come row by row, as they lie.
template <int D>
struct Block {
    uint8_t k[kBlock * D / 2];
    uint8_t v[kBlock * D / 2];
    float2 k_pair[kBlock][2];
    float2 v_pair[kBlock][2];
};

// The key of slot s (of 8) of a product's keys, and of slot s + 8: that key + 8.  The order is free; this one lets neither the
// reads of K (a lane a key's 16 or 8 bytes, eight lanes' keys together slots 2i, 2i + 1 or four) nor those of V (slots 0, 2, 4,
// 6 or 1, 3, 5, 7 together) meet a bank twice.
template <int D>
__device__ __forceinline__ int key_of_slot(int s) {
    return (int)((D == 128 ? 0x65742130u : 0x53427160u) >> (4 * s)) & 7;
}

// of byte c of row r of K or V in a block
template <int D>
__device__ __forceinline__ int place(int r, int c, bool swizzled) {
    return r * (D / 2) + (D == 128 && swizzled ? c ^ ((r >> 1 & 3) << 4) : c);
}

template <int N>
__device__ __forceinline__ void words(uint32_t (&x)[N], const uint8_t* p) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        x[0] = v.x;
        x[1] = v.y;
    } else {
        x[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// keys of the block at pos without a row (not in `valid`): flagged where one of the n tile rows from packed row m0 on sees it
__device__ __noinline__ void flag_lost(const DenseArgs& a, const Geom& g, int b, int64_t m0, int n, int n_kv, int pos, uint32_t valid) {
    const int lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
    if ((valid >> lane) & 1u) return;
    for (int r = 0; r < n; ++r) {
        const Interval iv = row_interval(g, a.mods, (int64_t)b * g.T + (m0 + r) / G, b, n_kv);
        if (pos + lane >= iv.lo && pos + lane < iv.hi) {
            flag(g.status, IDX_ERR_DEVICE_BOUNDS);
            return;
        }
    }
}

// What the products hold.  A weight goes with its value's scale, p s <= 2^15 with p <= 2^64 (see the running maximum): V's scales
// from 2^-57 on, or 0, keep every bit of both, and up to 2^32 neither the sum of the weights nor that of the minimums leaves f32.
// Scores are products of a key's scale and sum, q's unit and the call's scale, one after the other: each at most 2^60 (few_rows)
// has room.  Pieces of rows that see a key beyond that are done by rows_by_key.
constexpr float kMost = 0x1p32f, kMostScale = 0x1p60f;
constexpr int kMostUnit = 60;

__device__ __forceinline__ bool beyond(float2 k, float2 v) {
    constexpr uint32_t kLeast = 0x23000000u;      // 2^-57
    return fmaxf(fmaxf(fabsf(k.x), fabsf(k.y)), fmaxf(fabsf(v.x), fabsf(v.y))) > kMost || 2u * __float_as_uint(v.x) - 1u < 2u * kLeast - 1u;
}

// The rows of a CTA's piece, keys [j0, j1), key by key and all in f32: a warp to a row, a lane to D / 32 columns.  Results go
// where the first warp's would have gone (o_s, ml, low).
template <typename T, int D, int R>
__device__ __noinline__ void rows_by_key(const DenseArgs& a, const Geom& g, int b, int gkv, int64_t m0, int n_rows, int n_kv, int j0, int j1,
                                         float* o_s, int pitch, float2* ml, float* low) {
    constexpr int C = D / 32;
    const int lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
    for (int r = threadIdx.x >> 5; r < R; r += kWarps) {
        float M = -INFINITY, l = 0.f, acc[C];
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = 0.f;
        if (r < n_rows) {
            const int64_t row = (int64_t)b * g.T + (m0 + r) / G;
            const int h = gkv * G + (int)((m0 + r) % G);
            const Interval iv = row_interval(g, a.mods, row, b, n_kv);
            const T* q = static_cast<const T*>(a.q) + (row * a.Hq + h) * D + lane * C;
            const float slope = a.mods.slopes ? a.mods.slopes[h] : 0.f;
            const int end = min(iv.hi, j1);
            for (int j = max(iv.lo, j0); j < end; ++j) {
                const int64_t at = key_row(g, b, j);
                if (at < 0 || at >= a.kv_rows) continue;      // (flagged when its block came)
                auto load = [&](const void* cache, int64_t stride, float (&y)[C]) {
                    const uint8_t* p = static_cast<const uint8_t*>(cache) + at * stride;
                    const float2 pair = reinterpret_cast<const float2*>(p + a.Hkv * (D / 2))[gkv];
                    const uint8_t* c = p + gkv * (D / 2) + lane * (C / 2);
                    const uint32_t n = C == 4 ? *reinterpret_cast<const uint16_t*>(c) : *c;
#pragma unroll
                    for (int i = 0; i < C; ++i) y[i] = fmaf((float)((n >> (4 * i)) & 15u), pair.x, pair.y);
                };
                float k[C], v[C], x = 0.f;
                load(a.k, a.k_stride, k);
                load(a.v, a.v_stride, v);
#pragma unroll
                for (int i = 0; i < C; ++i) x = fmaf(to_f32(q[i]), k[i], x);
#pragma unroll
                for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                x *= a.scale;
                if (a.mods.softcap > 0.f) x = a.mods.softcap * tanhf(x / a.mods.softcap);
                x = (x - slope * fabsf((float)(iv.pos - j))) * kLog2e;
                if (x == -INFINITY) continue;
                const float top = fmaxf(M, x), al = exp2f(M - top), w = exp2f(x - top);
                M = top;
                l = fmaf(l, al, w);
#pragma unroll
                for (int i = 0; i < C; ++i) acc[i] = fmaf(acc[i], al, w * v[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < C; ++i) o_s[r * pitch + lane * C + i] = acc[i];
        if (lane < kWarps) ml[lane * R + r] = lane ? make_float2(0.f, 0.f) : make_float2(M, l);
        if (lane == 0) low[r] = 0.f;
    }
}

template <int D, int NB>
struct Shape {
    static constexpr int R = 8 * NB;
    static constexpr int kStages = NB == 1 ? 2 : 3;
    static constexpr int kCtas = NB == 1 ? 3 : 2;
    static constexpr int kRing = (int)sizeof(Block<D>) * kStages * kWarps;
    static constexpr int kPitch = D + 4;                              // the warps' results, over the rings
    static constexpr int kBytes = 1024 + (kRing > kWarps * R * kPitch * 4 ? kRing : kWarps * R * kPitch * 4);
};

template <typename T, int D, int NB, bool kMods>
__global__ void __launch_bounds__(kThreads, Shape<D, NB>::kCtas)
    q4_kernel(const __grid_constant__ Q4Args p, const __grid_constant__ Geom g, const __grid_constant__ Maps maps) {
    using S = Shape<D, NB>;
    constexpr int R = S::R;
    constexpr bool kRest = std::is_same<T, __half>::value;      // the weights in two parts
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kWarps][S::kStages];
    __shared__ float2 ml_s[kWarps][R];               // maximum, sum
    __shared__ float low_s[kWarps][R];               // sum of weight * m'
    __shared__ uint32_t valid_s[kWarps][S::kStages]; // keys of a block that have a row
    __shared__ int wide_s[kWarps];                   // whether numbers came that the products do not hold
    static_assert(kWarps == 4, "four marks");
    float* o_s = reinterpret_cast<float*>(smem);     // [warp][R][kPitch]
    const DenseArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const int G = a.Hq / a.Hkv;
    const int columns = a.Hkv * p.row_tiles;
    if (p.part_o) pdl_trigger();     // (the merge follows)
    if (lane == 0) {
        wide_s[warp] = 0;
        for (int i = 0; i < S::kStages; ++i) mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    const int col = (int)(blockIdx.x % columns);
    const Cut cut = cut_of(g, p, (int)(blockIdx.x / columns), true);
    if (cut.b < 0) return;
    const int gkv = col % a.Hkv, b = cut.b;
    const int64_t m0 = (int64_t)(col / a.Hkv) * R;
    const int n_rows = (int)min((int64_t)g.T * G - m0, (int64_t)R);
    const int n_kv = seq_n_kv(g, b);
    const int t00 = (int)(m0 / G), h00 = (int)(m0 - (int64_t)t00 * G);
    auto row_of = [&](int r, int& h) {       // batch row and head of the tile's row r
        const int t = (h00 + r) / G;
        h = gkv * G + h00 + r - t * G;
        return (int64_t)b * g.T + t00 + t;
    };

    // ---- the rows that this lane's scores belong to: 8 nb + 2 tq and the next
    int lo[NB][2], hi[NB][2];
    float d0[NB][2], slope[NB][2];     // own position, bias
    int k0 = INT32_MAX, k1 = 0, full0 = 0, full1 = INT32_MAX;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * nb + 2 * tq + e;
            Interval iv = {0, 0, 0};
            slope[nb][e] = 0.f;
            if (r < n_rows) {
                int h;
                const int64_t row = row_of(r, h);
                iv = row_interval(g, a.mods, row, b, n_kv);
                if (kMods && a.mods.slopes) slope[nb][e] = a.mods.slopes[h] * kLog2e;
            }
            lo[nb][e] = iv.lo;
            hi[nb][e] = iv.hi;
            d0[nb][e] = (float)iv.pos;
            if (iv.lo < iv.hi) {       // (a row that sees nothing takes what it gets and writes zeros)
                k0 = min(k0, iv.lo);
                k1 = max(k1, iv.hi);
                full0 = max(full0, iv.lo);
                full1 = min(full1, iv.hi);
            }
        }
    k0 = __reduce_min_sync(0xffffffffu, k0);
    k1 = __reduce_max_sync(0xffffffffu, k1);
    full0 = __reduce_max_sync(0xffffffffu, full0);
    full1 = __reduce_min_sync(0xffffffffu, full1);
    int blocks = 0, base = 0;       // this CTA's blocks of 32 keys, from position `base`
    if (k0 < k1) {
        const int first = k0 / kBlock, n = (k1 + kBlock - 1) / kBlock - first;
        const int share = (n + cut.pieces - 1) / cut.pieces;
        const int64_t from = (int64_t)cut.piece * share;
        blocks = (int)max(min((int64_t)share, n - from), (int64_t)0);
        base = blocks ? (int)((first + from) * kBlock) : 0;
    }

    // ---- q: f16 at a power of two of the row's, laid out as K's codes lie; its sum
    uint32_t qf[NB][D / 16][2];
    float unit[NB][2], qsum[NB][2], qodd[NB][2];      // of this lane's score rows
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        float x[D / 4];
        const int r = 8 * nb + gq;
        int h = 0;
        const int64_t row = r < n_rows ? row_of(r, h) : 0;
        const T* q = static_cast<const T*>(a.q) + (row * a.Hq + h) * D + tq * (D / 4);
        float big = 0.f, sum = 0.f, odd = 0.f;
#pragma unroll
        for (int c = 0; c < D / 4; c += 8) {
            T y[8];
            *reinterpret_cast<uint4*>(y) = r < n_rows ? *reinterpret_cast<const uint4*>(q + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[c + i] = to_f32(y[i]);
                big = fmaxf(big, fabsf(x[c + i]));
                sum += x[c + i];
                if (i & 1) odd += x[c + i];
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            odd += __shfl_xor_sync(0xffffffffu, odd, o);
        }
        // 2^e with big / 2^e in [2^9, 2^10) (1 for a row of zeros or of no numbers; e kept where 2^e and 2^-e are normal)
        const int e = big > 0.f && big < INFINITY ? min(max((int)(__float_as_uint(big) >> 23) - 127 - 9, -126), 126) : 0;
        if (e > kMostUnit) wide_s[warp] = 1;
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                qf[nb][2 * w + i / 2][i & 1] =
                    h2(__floats2half2_rn(x[8 * w + i] * (i & 1 ? inv * 0.0625f : inv), x[8 * w + i + 4] * (i & 1 ? inv * 0.0625f : inv)));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            unit[nb][s] = __shfl_sync(0xffffffffu, up, (2 * tq + s) * 4);
            qsum[nb][s] = __shfl_sync(0xffffffffu, sum, (2 * tq + s) * 4);
            qodd[nb][s] = __shfl_sync(0xffffffffu, odd * inv, (2 * tq + s) * 4) * -kOdd;
        }
    }

    // ---- the blocks' way to shared memory: a lane looks up its key's row, the first lane of each box asks for it
    Block<D>* ring = reinterpret_cast<Block<D>*>(smem) + warp * S::kStages;
    const int32_t* table = g.page_table ? g.page_table + (int64_t)b * g.page_table_stride : nullptr;
    const int kv_rows = (int)a.kv_rows, size = table ? g.page_size : 0;
    const int row0 = table ? 0 : (int)max(min(seq_row0(g, b), a.kv_rows), (int64_t)INT32_MIN);
    // the page of this lane's key of a block, and the row within it (asked for a block ahead of its bytes)
    struct Place {
        int page, in;
    };
    auto place_of = [&](int blk) -> Place {
        const int j = base + blk * kBlock + lane;
        if (blk >= blocks || j >= k1) return {-1, 0};
        if (!table) return {0, j};
        const int pg = p.shift >= 0 ? j >> p.shift : j / size;
        return {table[pg], j - pg * size};
    };
    auto fetch = [&](int blk, int stage, Place at_page) {
        if (blk >= blocks) return;
        // (32 bits hold the row of a page that there is)
        const bool there = table ? (uint32_t)at_page.page < p.pages : at_page.page == 0;
        const int row = at_page.page * size + row0 + at_page.in;
        const uint32_t valid = __ballot_sync(0xffffffffu, there && (uint32_t)row < (uint32_t)kv_rows);
        // (what is past the last key, or out of range, is filled with zeros: a row behind the cache.  A box may start before it.)
        const int at = there && row > -kBlock && row < kv_rows ? row : kv_rows;
        Block<D>& to = ring[stage];
        uint64_t* bar = &full[warp][stage];
        if (lane == 0) {
            valid_s[warp][stage] = valid;
            mbar_arrive_expect_tx(bar, p.box ? (uint32_t)sizeof(Block<D>) : (uint32_t)(__popc(valid) * (D + 32)));
        }
        __syncwarp();
        if (p.box) {
            if ((lane & (p.box - 1)) == 0) {
                tma_load_3d(to.k + lane * (D / 2), &maps.k, bar, 0, gkv, at);
                tma_load_3d(to.v + lane * (D / 2), &maps.v, bar, 0, gkv, at);
                tma_load_3d(to.k_pair[lane], &maps.k_pair, bar, (gkv >> 1) * 16, 0, at);
                tma_load_3d(to.v_pair[lane], &maps.v_pair, bar, (gkv >> 1) * 16, 0, at);
            }
        } else if ((valid >> lane) & 1u) {     // (what stays of an earlier block is masked)
            const uint8_t* kr = static_cast<const uint8_t*>(a.k) + (int64_t)row * a.k_stride;
            const uint8_t* vr = static_cast<const uint8_t*>(a.v) + (int64_t)row * a.v_stride;
            const int pair = a.Hkv * (D / 2) + (gkv >> 1) * 16;
            bulk_load(to.k + lane * (D / 2), kr + gkv * (D / 2), D / 2, bar);
            bulk_load(to.v + lane * (D / 2), vr + gkv * (D / 2), D / 2, bar);
            bulk_load(to.k_pair[lane], kr + pair, 16, bar);
            bulk_load(to.v_pair[lane], vr + pair, 16, bar);
        }
    };

    float o[NB][D / 16][4];
    // m: the rows' running maximum (log2 units, 0 while there is none), less kShift; top: what a weight times its scale may be
    float m[NB][2], l_run[NB][2], low_run[NB][2];
    __half2 top[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nb][i][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[nb][e] = l_run[nb][e] = low_run[nb][e] = 0.f;
        }
        top[nb] = __float2half2_rn(-1.f);
    }
    const float c = a.scale * kLog2e;
    const float cap = a.mods.softcap, inv_cap = cap > 0.f ? a.scale / cap : 0.f;

    const uint8_t* my_ring = reinterpret_cast<const uint8_t*>(ring);
    const int kq = key_of_slot<D>(gq);       // key of this lane's scores (and + 8)
    const int k_off = place<D>(kq, tq * (D / 8), p.box != 0), pair_off = kBlock * D + kq * 16 + (gkv & 1) * 8;
    const int v_off[2] = {kBlock * D / 2 + place<D>(key_of_slot<D>(2 * tq), gq * (D / 16), p.box != 0),
                          kBlock * D / 2 + place<D>(key_of_slot<D>(2 * tq + 1), gq * (D / 16), p.box != 0)};

    // (two of it: where every row sees every key of a block nothing is masked)
    auto compute = [&](auto all, int stage, int key0, uint32_t valid) {
        constexpr bool whole = decltype(all)::value;
        const uint8_t* x = my_ring + stage * (int)sizeof(Block<D>);
        float s[2][NB][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t k[2][D / 32];
            words(k[0], x + k_off + h * 8 * D);
            words(k[1], x + k_off + h * 8 * D + 4 * D);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                uint32_t c0[4], c1[4];
                codes<true>(k[0][w], c0);
                codes<true>(k[1][w], c1);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if (w == 0)
                        mma_from(s[h][nb], c0[0], c1[0], c0[1], c1[1], qf[nb][0][0], qf[nb][0][1], qodd[nb][0], qodd[nb][1]);
                    else
                        mma(s[h][nb], c0[0], c1[0], c0[1], c1[1], qf[nb][2 * w][0], qf[nb][2 * w][1]);
                    mma(s[h][nb], c0[2], c1[2], c0[3], c1[3], qf[nb][2 * w + 1][0], qf[nb][2 * w + 1][1]);
                }
            }
        }
        // scores in log2 units, less m: element e of half h is key 16 h + 8 (e / 2) + gq, row 8 nb + 2 tq + e % 2
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 pr = *reinterpret_cast<const float2*>(x + pair_off + (16 * h + 8 * k) * 16);
                const float ks = kMods ? pr.x : pr.x * c, km = fmaf(8.f, pr.x, pr.y) * (kMods ? 1.f : c);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float y = s[h][nb][2 * k + r] * unit[nb][r];
                        if (kMods) {
                            y = fmaf(km, qsum[nb][r], ks * y);
                            if (cap > 0.f) {
                                const float z = y * inv_cap, zz = z * z;
                                // (tanh's series where the other form cancels; the next term is below 2^-24 of it)
                                const float near = z * fmaf(fmaf(fmaf(fmaf(62.f / 2835.f, zz, -17.f / 315.f), zz, 2.f / 15.f), zz, -1.f / 3.f), zz, 1.f);
                                y = cap * kLog2e * (fabsf(z) > 0.3f ? tanh_large(z) : near);
                            } else {
                                y *= c;
                            }
                            y = fmaf(-slope[nb][r], fabsf(d0[nb][r] - (float)(key0 + 16 * h + 8 * k + kq)), y) - m[nb][r];
                        } else {
                            y = fmaf(ks, y, fmaf(km, qsum[nb][r], -m[nb][r]));
                        }
                        s[h][nb][2 * k + r] = y;
                    }
            }
        if (!whole) {
            const uint32_t v = valid >> kq;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 16 * h + 8 * (e >> 1), key = key0 + j + kq;
                        if (!((v >> j) & 1u) || key < lo[nb][e & 1] || key >= hi[nb][e & 1]) s[h][nb][e] = -INFINITY;
                    }
            if (valid != ~0u) flag_lost(a, g, b, m0, n_rows, n_kv, key0, valid);
        }
        float2 vp[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) vp[h][k] = *reinterpret_cast<const float2*>(x + pair_off + kBlock * 16 + (16 * h + 8 * k) * 16);
        // (each lane looks at one key's; 66.3 us without, 67.3 with, of 16 sequences of up to 32768 keys)
        const int own = kq + 8 * tq;
        const float2 own_k = *reinterpret_cast<const float2*>(x + pair_off + 8 * 16 * tq);
        const float2 own_v = *reinterpret_cast<const float2*>(x + pair_off + 8 * 16 * tq + kBlock * 16);
        if ((whole || (((valid >> own) & 1u) && key0 + own >= k0)) && beyond(own_k, own_v)) wide_s[warp] = 1;
        float pr[2][NB][4], sum[NB][2];
        uint32_t wh[2][NB][2];
        auto weigh = [&] {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float w[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int e = 2 * k + r;
                            pr[h][nb][e] = ex2_approx(s[h][nb][e]);
                            w[r] = pr[h][nb][e] * vp[h][k].x;
                            // (whatever the scale of a key that a row does not see)
                            if (!whole && s[h][nb][e] == -INFINITY) w[r] = 0.f;
                        }
                        wh[h][nb][k] = h2(__floats2half2_rn(w[0], w[1]));
                    }
#pragma unroll
                for (int r = 0; r < 2; ++r) sum[nb][r] = (pr[0][nb][r] + pr[0][nb][r + 2]) + (pr[1][nb][r] + pr[1][nb][r + 2]);
            }
        };
        weigh();
        // The maximum (of weight times scale, which is what is rounded to f16) follows lazily: a product stays below 2^15, kept
        // 2^7 larger than a weight of the largest, so that those down to 2^-31 of it are not lost in f16's subnormals; a
        // weight below 2^64, whatever its scale.
        bool rise = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            __half2 big = __habs2(as_h2(wh[0][nb][0]));
            big = __hmax2_nan(big, __habs2(as_h2(wh[0][nb][1])));
            big = __hmax2_nan(big, __hmax2_nan(__habs2(as_h2(wh[1][nb][0])), __habs2(as_h2(wh[1][nb][1]))));
            rise |= !__hble2(big, top[nb]);
#pragma unroll
            for (int r = 0; r < 2; ++r) rise |= !(sum[nb][r] <= 0x1p64f);
        }
        if (__any_sync(0xffffffffu, rise)) {
            float lg[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) lg[h][k] = fminf(fmaxf(lg2_approx(fabsf(vp[h][k].x)), kShift - 64.f), 127.f);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float by = fmaxf(fmaxf(s[0][nb][r] + lg[0][0], s[0][nb][r + 2] + lg[0][1]),
                                     fmaxf(s[1][nb][r] + lg[1][0], s[1][nb][r + 2] + lg[1][1])) - kShift;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) by = fmaxf(by, __shfl_xor_sync(0xffffffffu, by, d));
                    const bool first = (r ? __high2float(top[nb]) : __low2float(top[nb])) < 0.f;
                    if (by == -INFINITY || (!first && by < 0.f)) by = 0.f;
                    else if (first) top[nb] = r ? __halves2half2(__low2half(top[nb]), __float2half(32768.f))
                                                : __halves2half2(__float2half(32768.f), __high2half(top[nb]));
                    const float al = first ? 0.f : ex2_approx(-by);
                    m[nb][r] += by;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        s[h][nb][r] -= by;
                        s[h][nb][r + 2] -= by;
                    }
                    l_run[nb][r] *= al;
                    low_run[nb][r] *= al;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        o[nb][k][r] *= al;
                        o[nb][k][r + 2] *= al;
                    }
                }
            weigh();
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < 2; ++r) l_run[nb][r] += sum[nb][r];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t pf[NB][2], pr_rest[kRest ? NB : 1][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float low = fmaf(8.f, vp[h][k].x, vp[h][k].y);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float add[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        add[r] = low_run[nb][r];
                        low_run[nb][r] = fmaf(pr[h][nb][2 * k + r], low, low_run[nb][r]);
                    }
                    if (!whole) {
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            if (s[h][nb][2 * k + r] == -INFINITY) low_run[nb][r] = add[r];
                    }
                    pf[nb][k] = transpose8(wh[h][nb][k]);
                    if constexpr (kRest) {
                        const float2 w = __half22float2(as_h2(wh[h][nb][k]));
                        float rest[2] = {fmaf(pr[h][nb][2 * k], vp[h][k].x, -w.x), fmaf(pr[h][nb][2 * k + 1], vp[h][k].x, -w.y)};
                        if (!whole) {
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                if (s[h][nb][2 * k + r] == -INFINITY) rest[r] = 0.f;
                        }
                        pr_rest[nb][k] = transpose8(h2(__floats2half2_rn(rest[0], rest[1])));
                    }
                }
            }
            uint32_t v[4][D / 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) words(v[e], x + v_off[e & 1] + (16 * h + 8 * (e >> 1)) * (D / 2));
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                // halves of two keys side by side, then a column's code of both
                uint32_t f[4][4];
                codes<false>(__byte_perm(v[0][i], v[1][i], 0x5410), f[0]);
                codes<false>(__byte_perm(v[2][i], v[3][i], 0x5410), f[1]);
                codes<false>(__byte_perm(v[0][i], v[1][i], 0x7632), f[2]);
                codes<false>(__byte_perm(v[2][i], v[3][i], 0x7632), f[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int hh = k & 2, j = 2 * (k & 1);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        mma(o[nb][4 * i + k], f[hh][j], f[hh][j + 1], f[hh + 1][j], f[hh + 1][j + 1], pf[nb][0], pf[nb][1]);
                        if constexpr (kRest)
                            mma(o[nb][4 * i + k], f[hh][j], f[hh][j + 1], f[hh + 1][j], f[hh + 1][j + 1], pr_rest[nb][0], pr_rest[nb][1]);
                    }
                }
            }
        }
    };

    if (warp < blocks) {
        constexpr int kAhead = S::kStages - 1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(warp + i * kWarps, i, place_of(warp + i * kWarps));
        Place next = place_of(warp + kAhead * kWarps);
        int stage = 0, phase = 0, into = kAhead;
        for (int i = warp; i < blocks; i += kWarps) {
            __syncwarp();       // every lane is done with the block before, whose place is filled again
            fetch(i + kAhead * kWarps, into, next);
            next = place_of(i + (kAhead + 1) * kWarps);
            if (!warp_wait(&full[warp][stage], (uint32_t)phase)) {
                flag(g.status, IDX_ERR_TIMEOUT);
                // what is on its way lands before the place is used otherwise
                for (int k = i; k < blocks && k <= i + kAhead * kWarps; k += kWarps) {
                    warp_wait(&full[warp][stage], (uint32_t)phase);
                    if (++stage == S::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                break;
            }
            const int key0 = base + i * kBlock;
            const uint32_t valid = valid_s[warp][stage];
            if (valid == ~0u && key0 >= full0 && key0 + kBlock <= full1)
                compute(std::true_type{}, stage, key0, valid);
            else
                compute(std::false_type{}, stage, key0, valid);
            if (++stage == S::kStages) {
                stage = 0;
                phase ^= 1;
            }
            into = into + 1 == S::kStages ? 0 : into + 1;
        }
    }
    __syncthreads();       // the rings are done with

    // ---- the warps' results: sums over the lanes of a row, then over the warps
    if (wide_s[0] | wide_s[1] | wide_s[2] | wide_s[3]) {
        rows_by_key<T, D, R>(a, g, b, gkv, m0, n_rows, n_kv, base, base + blocks * kBlock, o_s, S::kPitch, &ml_s[0][0], low_s[0]);
    } else {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l_run[nb][e] += __shfl_xor_sync(0xffffffffu, l_run[nb][e], d);
                    low_run[nb][e] += __shfl_xor_sync(0xffffffffu, low_run[nb][e], d);
                }
                const int r = 8 * nb + 2 * tq + e;
                if (gq == 0) {
                    ml_s[warp][r] = make_float2(m[nb][e], l_run[nb][e]);
                    low_s[warp][r] = low_run[nb][e];
                }
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    *reinterpret_cast<float2*>(o_s + (warp * R + r) * S::kPitch + gq * (D / 8) + 2 * k) =
                        make_float2(o[nb][k][e], o[nb][k][e + 2]);
            }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n_rows * (D / 4); e += kThreads) {
        const int r = e / (D / 4), cc = e % (D / 4) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (ml_s[w][r].y != 0.f) M = fmaxf(M, ml_s[w][r].x);
        float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 ml = ml_s[w][r];
            if (ml.y == 0.f) continue;
            const float f = exp2f(ml.x - M);
            const float4 v = *reinterpret_cast<const float4*>(o_s + (w * R + r) * S::kPitch + cc);
            const float low = low_s[w][r];
            l = fmaf(f, ml.y, l);
            acc[0] = fmaf(f, v.x + low, acc[0]);
            acc[1] = fmaf(f, v.y + low, acc[1]);
            acc[2] = fmaf(f, v.z + low, acc[2]);
            acc[3] = fmaf(f, v.w + low, acc[3]);
        }
        int h;
        const int64_t row = row_of(r, h);
        const Interval iv = row_interval(g, a.mods, row, b, n_kv);
        if (iv.lo >= iv.hi) l = 0.f;
        if (p.part_o) {
            const int64_t at = (int64_t)blockIdx.x * R + r;
            *reinterpret_cast<float4*>(p.part_o + at * D + cc) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (cc == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(M, l);
        } else {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            T y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = from_f32<T>(l == 0.f ? 0.f : acc[i] * inv);
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (row * a.Hq + h) * D + cc) = *reinterpret_cast<const uint2*>(y);
            if (cc == 0 && a.lse) a.lse[row * a.Hq + h] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
        }
    }
}

// A CTA per packed row: its pieces shared by the warps, in a fixed order, four columns to a lane (heads of 64: half a warp to a
// piece) and kAtOnce pieces' loads on their way together.
constexpr int kMergeWarps = 16, kAtOnce = 4;

template <typename T, int D, int NB>
__global__ void __launch_bounds__(32 * kMergeWarps) q4_merge_kernel(Q4Args p, Geom g) {
    constexpr int R = 8 * NB, L = D / 4;       // lanes of a piece
    __shared__ float m_s[kMergeWarps * 2], l_s[kMergeWarps * 2];
    __shared__ __align__(16) float o_s[kMergeWarps * 2][D];
    const DenseArgs& a = p.a;
    const int lane = threadIdx.x % L, part = threadIdx.x / L, parts = blockDim.x / L;
    const int G = a.Hq / a.Hkv;
    const int rh = blockIdx.x, row = rh / a.Hq, h = rh - row * a.Hq, gkv = h / G, b = row / g.T;
    const int64_t m = (int64_t)(row - b * g.T) * G + h % G;
    pdl_wait();
    const Cut cut = cut_of(g, p, b, false);
    const int columns = a.Hkv * p.row_tiles;
    const int64_t first = ((int64_t)cut.first * columns + (m / R) * a.Hkv + gkv) * R + m % R, step = (int64_t)columns * R;
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = part * kAtOnce; s0 < cut.pieces; s0 += parts * kAtOnce) {
        float2 ml[kAtOnce];
        float4 x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t at = first + (int64_t)min(s0 + i, cut.pieces - 1) * step;
            ml[i] = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
            if (s0 + i >= cut.pieces) ml[i].y = 0.f;
            x[i] = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * lane);
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (ml[i].y != 0.f) top = fmaxf(top, ml[i].x);
        const float al = M == -INFINITY ? 0.f : exp2f(M - top);
        M = top;
        l *= al;
        acc = make_float4(acc.x * al, acc.y * al, acc.z * al, acc.w * al);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (ml[i].y == 0.f) continue;      // (a piece without keys)
            const float w = exp2f(ml[i].x - M);
            l = fmaf(w, ml[i].y, l);
            acc = make_float4(fmaf(w, x[i].x, acc.x), fmaf(w, x[i].y, acc.y), fmaf(w, x[i].z, acc.z), fmaf(w, x[i].w, acc.w));
        }
    }
    if (lane == 0) {
        m_s[part] = M;
        l_s[part] = l;
    }
    *reinterpret_cast<float4*>(&o_s[part][4 * lane]) = acc;
    __syncthreads();
    if (threadIdx.x >= D) return;
    const int used = min(parts, (cut.pieces + kAtOnce - 1) / kAtOnce);
    M = -INFINITY;
    for (int w = 0; w < used; ++w)
        if (l_s[w] != 0.f) M = fmaxf(M, m_s[w]);
    float den = 0.f, y = 0.f;
    for (int w = 0; w < used; ++w) {
        if (l_s[w] == 0.f) continue;
        const float f = exp2f(m_s[w] - M);
        den = fmaf(f, l_s[w], den);
        y = fmaf(f, o_s[w][threadIdx.x], y);
    }
    static_cast<T*>(a.out)[(int64_t)rh * D + threadIdx.x] = from_f32<T>(den == 0.f ? 0.f : y / den);
    if (threadIdx.x == 0 && a.lse) a.lse[rh] = den == 0.f ? -INFINITY : (M + log2f(den)) * kLn2;
}

size_t split_bytes(int64_t n_rows, int Hq, int dv) { return (size_t)n_rows * Hq * (dv + 2) * sizeof(float); }

int n_blocks(int64_t packed) { return packed <= 8 ? 1 : 2; }

// The pieces of all rows: as many as the SMs hold at once.  (Three times as many: 16 x 32768 keys 76 us for 65 with a packed row
// tile, 278 for 300 with four; one sequence of these 50 for 39.)
int slots_of(int nb) {
    int sms = sm_count();
    return (sms < 2 ? 152 : sms) * (nb == 1 ? Shape<128, 1>::kCtas : Shape<128, 2>::kCtas);
}

// CTAs of the few-rows kernel with pieces (0: one piece a row is as well)
int64_t piece_ctas(int64_t n_seq, int64_t columns, int64_t max_n_kv, int slots) {
    const int64_t by_keys = ((max_n_kv + kTile - 1) / kTile + kMinTiles - 1) / kMinTiles;
    if (by_keys <= 1 || n_seq * columns >= slots) return 0;
    const int64_t by_slots = slots / columns + n_seq;      // (each row's pieces are rounded up)
    return columns * (by_slots < n_seq * by_keys ? by_slots : n_seq * by_keys);
}

bool few_rows(const DenseArgs& a, int dtype, const Geom& g) {
    if (dtype == IDX_F32 || a.dk != a.dv || (a.dk != 64 && a.dk != 128)) return false;
    if (a.kv_rows < 1 || a.kv_rows > INT32_MAX - kBlock || g.max_n_kv > INT32_MAX - 2 * kBlock) return false;
    if (!(fabsf(a.scale) <= kMostScale)) return false;
    // (16 bytes of two heads' scales, which the last row may not have for the last of an odd number of heads; TMA's boxes do
    // without)
    if (g.page_table && box_rows(g.page_size, kBlock) < 8 && a.Hkv % 2) return false;
    const uint64_t all = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                         reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.k_stride | (uint64_t)a.v_stride;
    return all % 16 == 0;
}

template <typename T, int D, int NB>
cudaError_t go(const DenseArgs& a, const Geom& g, void* ws, size_t ws_bytes, cudaStream_t st) {
    constexpr int R = 8 * NB;
    const int64_t packed = (int64_t)g.T * (a.Hq / a.Hkv);
    Q4Args p = {};
    p.a = a;
    const int64_t tiles = (packed + R - 1) / R, columns = a.Hkv * tiles;
    if (columns * g.B > INT32_MAX / 2) return cudaErrorNotSupported;
    p.row_tiles = (int)tiles;
    p.pages = g.page_table ? (uint32_t)((a.kv_rows + g.page_size - 1) / g.page_size) : 0;
    p.box = box_rows(g.page_size, kBlock);
    if (p.box < 8) p.box = 0;
    const int box = p.box ? p.box : kBlock;
    p.shift = g.page_table && (g.page_size & (g.page_size - 1)) == 0 ? __builtin_ctz(g.page_size) : -1;
    Maps maps;
    const uint8_t *k = static_cast<const uint8_t*>(a.k), *v = static_cast<const uint8_t*>(a.v);
    const int64_t codes = (int64_t)a.Hkv * (D / 2);
    // (pairs of heads' scales; the last one of an odd number of heads is filled up with zeros)
    auto pairs = [&](CUtensorMap* m, const uint8_t* x, int64_t stride) {
        return make_q4_tmap(m, x + codes, a.Hkv * 8, 1, stride, stride, a.kv_rows, 16, box, false);
    };
    if (!make_q4_tmap(&maps.k, k, D / 2, a.Hkv, D / 2, a.k_stride, a.kv_rows, D / 2, box, D == 128) ||
        !make_q4_tmap(&maps.v, v, D / 2, a.Hkv, D / 2, a.v_stride, a.kv_rows, D / 2, box, D == 128) ||
        !pairs(&maps.k_pair, k, a.k_stride) || !pairs(&maps.v_pair, v, a.v_stride))
        return cudaErrorNotSupported;
    const int slots = slots_of(NB);
    int64_t ctas = piece_ctas(g.B, columns, g.max_n_kv, slots);
    if (ctas * R * (D + 2) * (int64_t)sizeof(float) > (int64_t)ws_bytes) ctas = 0;
    if (ctas) {
        p.slots = slots;
        p.part_o = static_cast<float*>(ws);
        p.part_ml = p.part_o + ctas * R * D;
    } else {
        ctas = columns * g.B;
    }
    const bool mods = a.mods.softcap > 0.f || a.mods.slopes;
    auto launch = [&](auto kern) {
        constexpr int bytes = Shape<D, NB>::kBytes;
        static_assert((bytes + 2048) * Shape<D, NB>::kCtas <= 233472, "shared memory of an SM");
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        return e != cudaSuccess ? e : launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), bytes, st, p, g, maps);
    };
    const cudaError_t e = mods ? launch(q4_kernel<T, D, NB, true>) : launch(q4_kernel<T, D, NB, false>);
    if (e != cudaSuccess || !p.part_o) return e;
    const int64_t n = (int64_t)g.B * g.T * a.Hq;
    // as many threads as the longest row's pieces may need, and as the columns of a row
    const int64_t most = std::min<int64_t>(slots / columns + 1, ((int64_t)g.max_n_kv + kTile * kMinTiles - 1) / (kTile * kMinTiles));
    int threads = (int)std::min<int64_t>((most + kAtOnce - 1) / kAtOnce * (D / 4), 32 * kMergeWarps);
    threads = std::max((threads + 31) / 32 * 32, D);
    return launch_pdl(q4_merge_kernel<T, D, NB>, dim3((unsigned)n), dim3(threads), 0, st, p, g);
}

// The positions that some row of a sequence sees, and nothing lost or found yet
__global__ void __launch_bounds__(256) span_kernel(idx_attn_mods mods, Geom g, int2* span, int* lost, int* top, int* k_top, int Hkv) {
    __shared__ int lo_s[8], hi_s[8];
    pdl_wait();
    const int b = blockIdx.x, warp = threadIdx.x >> 5;
    for (int h = threadIdx.x; h < Hkv; h += 256) {
        top[(int64_t)b * Hkv + h] = 0;
        if (k_top) k_top[(int64_t)b * Hkv + h] = 0;
    }
    const int n_kv = seq_n_kv(g, b);
    int lo = INT32_MAX, hi = 0;
    for (int t = threadIdx.x; t < g.T; t += 256) {
        const Interval iv = row_interval(g, mods, (int64_t)b * g.T + t, b, n_kv);
        if (iv.lo < iv.hi) {
            lo = min(lo, iv.lo);
            hi = max(hi, iv.hi);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if ((threadIdx.x & 31) == 0) {
        lo_s[warp] = lo;
        hi_s[warp] = hi;
    }
    __syncthreads();
    if (threadIdx.x) return;
    for (int i = 1; i < 8; ++i) {
        lo = min(lo, lo_s[i]);
        hi = max(hi, hi_s[i]);
    }
    span[b] = make_int2(lo, hi);
    if (b == 0) *lost = 0;
}

// The largest magnitude of V, and of K where k_top is given, in each (sequence, kv head)'s span, as a float's bits: what f16 is
// scaled by.  Values that are no numbers say nothing; numbers past f32's go the CUDA cores' way.  A maximum does not depend on the
// order.
constexpr int kTopKeys = 8;      // positions of a thread

__global__ void __launch_bounds__(256) top_kernel(ExpandArgs p, Geom g, int* top, int* k_top, int chunks) {
    pdl_wait();
    const ReadArgs& a = p.r;
    const int b = blockIdx.x / chunks, heads = min(a.Hkv, 256), at_once = 256 / heads;
    const int2 span = p.span[b];
    const int64_t first = (int64_t)(blockIdx.x - b * chunks) * (at_once * kTopKeys) + threadIdx.x / heads;
    if (threadIdx.x >= heads * at_once) return;
    for (int h = threadIdx.x % heads; h < a.Hkv; h += heads) {
        float most = 0.f, most_k = 0.f;
        auto take = [&](const void* cache, int64_t stride, int64_t row, int d, float& m) {
            const uint8_t* pairs = static_cast<const uint8_t*>(cache) + row * stride + a.Hkv * (d / 2);
            const float* pair = reinterpret_cast<const float*>(pairs) + 2 * h;
            const float scale = pair[0], low = pair[1];
            if (isfinite(scale) && isfinite(low)) m = fmaxf(m, fmaxf(fabsf(low), fabsf(fmaf(15.f, scale, low))));
        };
#pragma unroll
        for (int i = 0; i < kTopKeys; ++i) {
            const int64_t pos = first + i * at_once;
            if (pos < span.x || pos >= span.y) continue;
            const int64_t row = key_row(g, b, pos);
            if (row < 0 || row >= a.kv_rows) continue;
            take(a.v_cache, a.vc_stride, row, a.dv, most);
            if (k_top) take(a.k_cache, a.kc_stride, row, a.dk, most_k);
        }
        if (isinf(most) || isinf(most_k)) *p.lost = 1;
        auto put = [&](int* to, float m) {
            if (__float_as_int(m) > *(volatile int*)to) atomicMax(to, __float_as_int(m));
        };
        put(top + (int64_t)b * a.Hkv + h, most);
        if (k_top) put(k_top + (int64_t)b * a.Hkv + h, most_k);
    }
}

// where the expanded K (in two parts) and V (f16 calls: in two) lie in the workspace, behind the spans, the largest values and
// the mark of lost keys
struct Expanded {
    size_t top_at, k_top_at, k_at, rest_at, v_at, v_rest_at, bytes;
    Expanded(int dtype, int64_t n_seq, int64_t max_n_kv, int Hkv, int dk, int dv) {
        const size_t rows = (size_t)n_seq * max_n_kv * Hkv;
        top_at = n_seq * sizeof(int2) + sizeof(int);
        k_top_at = top_at + n_seq * Hkv * sizeof(int);      // (right behind, see DenseArgs)
        // (on whole lines: 16 bytes off them 4096 tokens on 12288 keys took 1070 us, 32 off 1025)
        auto line = [](size_t n) { return (n + 127) / 128 * 128; };
        k_at = line(k_top_at + n_seq * Hkv * sizeof(int));
        rest_at = line(k_at + rows * dk * 2);
        v_at = line(rest_at + rows * dk * 2);
        v_rest_at = line(v_at + rows * dv * 2);
        bytes = v_rest_at + (dtype == IDX_F16 ? rows * dv * 2 : 0);
    }
};

// Whether a call of these sizes expands K and V (given the workspace): where the codes would be expanded for many tiles of rows,
// or for heads that the few-rows kernel does not take; up to 64 GB of them (the bound max_n_kv counts, not what it turns out).
constexpr int64_t kMaxExpanded = (int64_t)1 << 36;

bool expands(int dtype, int64_t n_seq, int64_t packed, int64_t max_n_kv, int Hkv, int dk, int dv) {
    if (dtype == IDX_F32 || dk > 128 || dv > 128) return false;
    if (n_seq * max_n_kv > kMaxExpanded / (Hkv * (4 * (int64_t)dk + (dtype == IDX_F16 ? 4 : 2) * dv))) return false;
    return packed > kManyRows || dk != dv || (dk != 64 && dk != 128);
}

template <typename T>
cudaError_t run_few(const DenseArgs& a, const Geom& g, void* ws, size_t ws_bytes, cudaStream_t st) {
    const bool one = n_blocks((int64_t)g.T * (a.Hq / a.Hkv)) == 1;
    if (a.dk == 64) return one ? go<T, 64, 1>(a, g, ws, ws_bytes, st) : go<T, 64, 2>(a, g, ws, ws_bytes, st);
    return one ? go<T, 128, 1>(a, g, ws, ws_bytes, st) : go<T, 128, 2>(a, g, ws, ws_bytes, st);
}

}  // namespace

size_t q4_attn_workspace_bytes(int dtype, int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv, int dk, int dv) {
    if (expands(dtype, n_seq, n_q * (Hq / Hkv), max_n_kv, Hkv, dk, dv)) return Expanded(dtype, n_seq, max_n_kv, Hkv, dk, dv).bytes;
    if (dtype != IDX_F32 && dk == dv && (dk == 64 || dk == 128)) {
        const int64_t packed = n_q * (Hq / Hkv);
        const int nb = n_blocks(packed);
        const int64_t columns = Hkv * ((packed + 8 * nb - 1) / (8 * nb));
        return (size_t)(piece_ctas(n_seq, columns, max_n_kv, slots_of(nb)) * 8 * nb * (dk + 2) * sizeof(float));
    }
    const int splits = dense_generic_splits(n_seq, n_q, max_n_kv, Hq, Hkv, dk, dv);
    return splits > kDenseCluster ? splits * split_bytes(n_seq * n_q, Hq, dv) : 0;
}

// K and V of the span that some row sees, expanded, then dense_attn's tensor-core kernel on them: V rounded to f16 (and the
// weights with it: bf16 for both leaves 4096 rows on 16384 keys with errors of 0.0029 of the result, 0.0017 is the result's
// own rounding) at a power of two, K as a sum of two of dtype (16 or 22 bits), since the log of the weights' sum is f32.  Of
// the 985 to 1000 us of 4096 tokens of 32 heads on 16384 keys the second product of K takes some 240 (K in bf16 alone: 740),
// spans, largest values and expansion of 16384 rows some 30.  (Scales applied to the products of exact codes, in the softmax: 1455 us; it is the
// softmax that the kernel waits for.)  For f16 results the weights and V are in two parts too (1560 us).
// f16 calls have K at a power of two too, which the call's scale takes back.
// What that kernel cannot know of or hold, keys without a row in the cache, numbers of K beyond bf16's, keys whose V is 2^-28 or
// less of the largest and, in f16 calls, whose K is 2^-17 or less, sends everything through the CUDA cores again, which skip and
// flag the first and hold the others in f32.
static cudaError_t run_expanded(DenseArgs a, int dtype, const Geom& g, uint8_t* ws, cudaStream_t st) {
    const Expanded e(dtype, g.B, g.max_n_kv, a.Hkv, a.dk, a.dv);
    int2* span = reinterpret_cast<int2*>(ws);
    int* lost = reinterpret_cast<int*>(ws + (size_t)g.B * sizeof(int2));
    DenseArgs d = a;
    d.k = ws + e.k_at;
    d.v = ws + e.v_at;
    d.k_stride = (int64_t)a.Hkv * a.dk;
    d.v_stride = (int64_t)a.Hkv * a.dv;
    d.kv_rows = (int64_t)g.B * g.max_n_kv;
    Geom flat = g;
    flat.page_table = nullptr;
    flat.page_size = 0;
    flat.kv_start = nullptr;
    flat.kv_seq_stride = g.max_n_kv;
    if (!dense_tc_supported(d, dtype, flat)) return cudaErrorNotSupported;
    // (key splits that are a cluster: no more workspace)
    int splits = dense_tc_splits(g.B, g.T, g.max_n_kv, a.Hq, a.Hkv);
    const int tiles = (g.max_n_kv + kDenseTcKeys - 1) / kDenseTcKeys;
    splits = splits < kDenseCluster ? splits : kDenseCluster;
    d.splits = splits < tiles ? splits : tiles;
    ExpandArgs x = {};
    x.r.k_cache = a.k;
    x.r.v_cache = a.v;
    x.r.kc_stride = a.k_stride;
    x.r.vc_stride = a.v_stride;
    x.r.kv_rows = a.kv_rows;
    x.r.Hkv = a.Hkv;
    x.r.dk = a.dk;
    x.r.dv = a.dv;
    x.r.k_out = ws + e.k_at;
    x.r.v_out = ws + e.v_at;
    x.span = span;
    x.lost = lost;
    x.k_rest = ws + e.rest_at;
    d.k_rest = x.k_rest;
    int* k_top = nullptr;
    if (dtype == IDX_F16) {
        d.v_rest = x.v_rest = ws + e.v_rest_at;
        x.k_top = k_top = reinterpret_cast<int*>(ws + e.k_top_at);
    }
    int* top = reinterpret_cast<int*>(ws + e.top_at);
    x.v_top = d.v_top = top;
    Geom all = g;
    all.T = g.max_n_kv;
    const int64_t chunk = 256 / std::min(a.Hkv, 256) * kTopKeys, chunks = (g.max_n_kv + chunk - 1) / chunk;
    if (chunks * g.B > INT32_MAX) return cudaErrorNotSupported;
    cudaError_t err = launch_pdl(span_kernel, dim3((unsigned)g.B), dim3(256), 0, st, a.mods, g, span, lost, top, k_top, a.Hkv);
    if (err == cudaSuccess) err = launch_pdl(top_kernel, dim3((unsigned)(chunks * g.B)), dim3(256), 0, st, x, g, top, k_top, (int)chunks);
    if (err == cudaSuccess) err = launch_expand_q4(x, dtype, all, st);
    if (err == cudaSuccess) err = launch_dense_tc(d, dtype, flat, st);
    if (err != cudaSuccess) return err;
    a.splits = 1;
    a.only_if = lost;
    return launch_dense_generic_q4(a, dtype, g, st);
}

cudaError_t launch_attn_q4(DenseArgs a, int dtype, const Geom& g, void* ws, size_t ws_bytes, cudaStream_t st) {
    if (g.max_n_kv > 0 && expands(dtype, g.B, (int64_t)g.T * (a.Hq / a.Hkv), g.max_n_kv, a.Hkv, a.dk, a.dv) &&
        ws_bytes >= Expanded(dtype, g.B, g.max_n_kv, a.Hkv, a.dk, a.dv).bytes) {
        const cudaError_t e = run_expanded(a, dtype, g, static_cast<uint8_t*>(ws), st);
        if (e != cudaErrorNotSupported) return e;
    }
    if (few_rows(a, dtype, g)) {
        const cudaError_t e = dtype == IDX_BF16 ? run_few<__nv_bfloat16>(a, g, ws, ws_bytes, st) : run_few<__half>(a, g, ws, ws_bytes, st);
        if (e != cudaErrorNotSupported) return e;
    }
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
