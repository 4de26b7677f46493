// Dense attention over (paged) caches on the 5th-generation tensor cores
// (dense_attn in lidx.h), for 16-bit K/V of at most 128 columns each.
//
// The T query rows and the G = Hq / Hkv heads that share a kv head are packed
// into rows m = t*G + h, 128 to a tile (the M side of the MMAs), so a K or V
// tile that is read once serves every head of the group.  A CTA owns kTiles
// such tiles of one (sequence, kv head) and one split of its keys, and
// walks it in tiles of 128 keys:
//     S = Q K^T       [128 x 128] f32 in TMEM     (Q, K from shared memory)
//     P = 2^(S*c - m) bf16/f16, written over S in TMEM, 64 keys at a time
//     O = O + P V     [128 x dv] f32 in TMEM      (P from TMEM, V from shared memory),
//                     64 keys at a time: the first half's product runs while the
//                     softmax is on the second half
// Warps 0-3: TMA producer, an MMA issuer per row tile, V inspector; then four
// softmax warps per row tile (thread = row = TMEM lane), which also write the
// output.  With two row tiles per CTA a K/V tile is read for 256 rows and the
// tensor core works on one tile while the other's softmax runs; with one (up to
// 48 packed rows: a decode step) two CTAs share an SM and the walk is bound by the
// stream of K and V.
//
// What the shape follows from, measured on a GB300: a 128 x 128 x 16 product takes
// 64 cycles (128 x 64 x 16 with both operands in shared memory 48, so scores are
// made for 128 keys at a time), the issuers' queue is short, and a softmax of 128
// rows x 64 keys takes 650 to 800 cycles.  On 4096 rows x 16384 keys (32 / 4 heads
// of 128, causal): one issuer, a lane on its own 1.17 ms; the warp together 0.99;
// an issuer per row tile 0.80 (64-key scores, double buffered); this form 0.74.
//
// A row's maximum follows its scores lazily: O is rescaled (by the softmax
// warps, in TMEM) only when a score passes it by 2^8, so P stays <= 2^8.
// f16 weights are kept 2^7 larger still, so that weights down to 2^-31 of the
// largest are not lost in f16's subnormals.  P is rounded to the inputs' type
// for the second product (an error of half a step, averaged over the keys); its
// sum, the maxima and O stay f32.
//
// Masks are intervals: a tile that every row of a warp sees whole skips them.
// A tile that some row sees in part is looked over before its PV product: V rows
// that nobody sees (a page's unwritten end) are zeroed in shared memory, and a
// NaN or infinity in any other row of it - 0 times which would reach rows that
// do not see it - sends the CTA's rows to a scalar loop over their own keys,
// as does a page number out of range.
// Every wait is bounded; a timeout records IDX_ERR_TIMEOUT and the CTA winds down.
#include "dense_attn.cuh"
#include "sm100_ptx.cuh"

namespace lidx {
namespace {
using namespace sm100;

constexpr int kKeys = 128;             // keys per K/V tile
constexpr int kHalf = 64;              // keys per softmax step and second product
constexpr int kRows = 128;             // packed query rows per row tile
constexpr int kColBlock = 128 * 128;   // 64 columns x 128 rows of a tile, in the 128-byte swizzle
constexpr int kFewRows = 48;           // packed rows up to which a CTA has one row tile and half an SM
constexpr int kOtherWarps = 4;

// Scores of 64 keys in two buffers per row tile instead of 128 in one: S of the next step is made while the softmax is
// on this one.  It costs the tensor pipe a fifth (see above), so it is for where the softmax takes longer than the
// products: capped or biased scores, and narrow heads.  (A decode step's CTA, one row tile and bound by its loads: 150 us
// with one buffer, 156 with two.)
template <int D, bool kMods>
constexpr bool kDoubleS = kMods || D == 64;

// kTwo (see the kernel): a key tile is two entries of K's ring; kBoth: and two of V's
template <int D, int kTiles, bool kTwo = false, bool kBoth = false>
struct Cfg {
    static constexpr int kTileBytes = kKeys * D * 2;
    // rows of Q kept per row tile.  With kFewRows the M = 128 products read on into the K tile: what they
    // make of it stays in TMEM lanes that nobody reads.
    static constexpr int kQRows = kTiles == 2 ? kRows : kFewRows;
    static constexpr int kQTile = kQRows * D * 2;
    static constexpr int kQBlock = kQRows * 128;      // 64 columns of it
    static constexpr int kStagesK = kTwo ? (kTiles == 2 || D == 64 ? 3 : kBoth ? 1 : 2) : kTiles == 2 ? 2 : D == 64 ? 2 : 1;
    static constexpr int kStagesV = kTwo && D == 128 ? (kTiles == 2 || kBoth ? 2 : 1) : kTiles == 2 ? 3 : D == 64 ? 3 : 2;
    static constexpr int kCtas = kTiles == 2 ? 1 : 2;   // (two: 128 registers; with options 28 to 40 bytes are spilled)
    static constexpr int kKOff = kTiles * kQTile;
    static constexpr int kVOff = kKOff + kStagesK * kTileBytes;
    static constexpr int kCtlOff = kVOff + kStagesV * kTileBytes;
    // merged splits: the rows' results over the rings, then their maxima (log2 units) and sums
    static constexpr int kMergeRows = kTiles * ((kQRows + 31) / 32 * 32);
    static constexpr int kMlOff = kMergeRows * D * 4;
    static_assert(kMlOff + kMergeRows * 8 <= kCtlOff, "rows kept for the merge");
    static constexpr int kThreads = 32 * kOtherWarps + kRows * kTiles;
    static constexpr int kTmemCols = kTiles == 2 ? 512 : 256;
    static constexpr int kOCol = kTiles * kKeys;      // S of row tile i at i*kKeys, O at kOCol + i*D
};

struct Ctl {
    uint64_t kfull[3], kempty[3];
    uint64_t vfull[3], vempty[3];
    uint64_t vok[3];              // V looked over
    uint64_t sfull[2][2];         // S of a row tile written; one buffer: [i][0], and its PV products before are complete;
                                  // two: and those of two steps before
    uint64_t pready[2][2];        // a half of P written over it, O rescaled
    uint64_t pvdone[2];           // the first half's PV product complete
    uint64_t odone[2];            // every product of a row tile complete
    uint64_t done[2];
    uint32_t tmem_base;
    int abort;
    int dirty;                    // a NaN or infinity in a V row that only some rows see, or a page out of range
    int k0, k1, full0, full1;     // the CTA's keys, and those that each of its rows sees
};

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);   // two rounded to T
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 x = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}

struct TcArgs {
    DenseArgs a;
    int tiles;        // groups of kTiles row tiles per (sequence, kv head)
    int box;          // rows per TMA box: 128, or the largest power of two that divides the page
};

// A row's attention key by key, for the thread that owns it: the rare way, see the top.  q, K and V as stored, f32
// sums.  acc gets the unnormalised values, ml the maximum (log2 units) and the sum.
template <typename T, typename V>
__device__ __noinline__ void scalar_row(const DenseArgs& a, const Geom& g, int b, int gkv, int64_t rh, int h, Interval iv,
                                        int64_t s0, int64_t s1, float* acc, float* ml) {
    const T* q = static_cast<const T*>(a.q) + rh * a.dk;
    for (int c = 0; c < a.dv; ++c) acc[c] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int64_t lo = iv.lo > s0 ? iv.lo : s0, hi = iv.hi < s1 ? iv.hi : s1;
    for (int64_t j = lo; j < hi; ++j) {
        const int64_t row = key_row(g, b, j);
        if (row < 0 || row >= a.kv_rows) {
            flag(g.status, IDX_ERR_DEVICE_BOUNDS);
            continue;
        }
        const T* k = static_cast<const T*>(a.k) + row * a.k_stride + (int64_t)gkv * a.dk;
        const V* v = static_cast<const V*>(a.v) + row * a.v_stride + (int64_t)gkv * a.dv;
        const T* rest = a.k_rest ? static_cast<const T*>(a.k_rest) + row * a.k_stride + (int64_t)gkv * a.dk : nullptr;
        const V* v_rest = a.v_rest ? static_cast<const V*>(a.v_rest) + row * a.v_stride + (int64_t)gkv * a.dv : nullptr;
        float x = 0.f;
        for (int c = 0; c < a.dk; ++c) x = fmaf(to_f32(q[c]), to_f32(k[c]) + (rest ? to_f32(rest[c]) : 0.f), x);
        x *= a.v_rest ? a.scale * exp2_whole(k_exponent(a.v_top[(int64_t)(g.B + b) * a.Hkv + gkv])) : a.scale;
        if (a.mods.softcap > 0.f) x = a.mods.softcap * tanhf(x / a.mods.softcap);
        if (a.mods.slopes) x -= a.mods.slopes[h] * fabsf((float)(iv.pos - j));
        x *= kLog2e;
        const float mn = fmaxf(m, x);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float al = m == mn ? 1.f : exp2f(m - ref);
        const float w = exp2f(x - ref);
        m = mn;
        l = fmaf(l, al, w);
        for (int c = 0; c < a.dv; ++c) acc[c] = fmaf(w, to_f32(v[c]) + (v_rest ? to_f32(v_rest[c]) : 0.f), al == 1.f ? acc[c] : acc[c] * al);
    }
    ml[0] = m;
    ml[1] = l;
}

// 32 columns of a row into its warp's staging rows of W columns (16-byte pieces, swizzled by the row)
template <typename E, int W>
__device__ __forceinline__ void stage_cols(uint8_t* rows, int row, int c0, const float (&v)[32]) {
    constexpr int kPer = 16 / (int)sizeof(E);
    uint8_t* r = rows + row * (W * (int)sizeof(E));
#pragma unroll
    for (int i = 0; i < 32 / kPer; ++i) {
        uint4 x;
        if constexpr (sizeof(E) == 4)
            x = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                           __float_as_uint(v[4 * i + 3]));
        else
            x = make_uint4(pack2<E>(v[8 * i], v[8 * i + 1]), pack2<E>(v[8 * i + 2], v[8 * i + 3]),
                           pack2<E>(v[8 * i + 4], v[8 * i + 5]), pack2<E>(v[8 * i + 6], v[8 * i + 7]));
        *reinterpret_cast<uint4*>(r + (((c0 / kPer + i) ^ (row & 7)) << 4)) = x;
    }
}

// the first n columns of the warp's first n_rows staged rows to out (row r at out + at_r, elements), whole rows at a
// time
template <typename E, int W>
__device__ __forceinline__ void store_rows(E* out, int64_t at, int n_rows, const uint8_t* rows, int n) {
    constexpr int kPer = 16 / (int)sizeof(E);
    const int lane = threadIdx.x & 31;
    auto piece = [&](int row, int pc, bool ok) {
        const int64_t to = __shfl_sync(0xffffffffu, at, row);
        if (ok)
            *reinterpret_cast<uint4*>(out + to + pc * kPer) =
                *reinterpret_cast<const uint4*>(rows + row * (W * (int)sizeof(E)) + ((pc ^ (row & 7)) << 4));
    };
    __syncwarp();
    if (n == W) {
        constexpr int kPieces = W / kPer, kStep = 32 / kPieces;    // rows per instruction
        static_assert(32 % kPieces == 0, "whole rows");
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += kStep) {
            if (r0 >= n_rows) break;
            const int row = r0 + lane / kPieces;
            piece(row, lane % kPieces, row < n_rows);
        }
    } else {
        const int pieces = n / kPer;
        for (int e = lane; e - lane < n_rows * pieces; e += 32) {
            const int row = e / pieces;
            piece(row & 31, e - row * pieces, row < n_rows);
        }
    }
    __syncwarp();
}

// kTwo: K is the sum of two tensors of T, for keys that T alone does not hold (values of 4-bit codes): the scores are two
// products into the same accumulators.  V and the weights are f16 then, V at a power of two.  4096 tokens of 32 heads of 128 on
// 16384 keys: 965 us, tensor pipe busy on 74 % of the active cycles (57 % with K in one part).
// With f16 q the results are f16 too, and roundings of V and of the weights would be as large as the results' own: both are in
// two parts as well (kBoth), P's second one beside the first in TMEM, and O three products: with one part each results were off by
// 1.7 times their rounding.  The same tokens take 1518 us, tensor pipe 81 %.  With one row tile of heads above 64 columns K's
// parts share a place, so that two CTAs still share an SM: 16 sequences of up to 32768 keys, 20 heads of 80 on 4, with the
// expansion 665 us (527 in bf16, with one part each; an SM to itself and three places 747, but one such sequence 126 for 154).
template <typename T, bool kTwo>
constexpr bool kBothParts = kTwo && std::is_same<T, __half>::value;

template <typename T, int D, int kTiles, bool kTwo>
using CfgOf = Cfg<D, kTiles, kTwo, kBothParts<T, kTwo>>;

template <typename T, int D, int kTiles, bool kMods, bool kTwo>
__global__ void __launch_bounds__(CfgOf<T, D, kTiles, kTwo>::kThreads, CfgOf<T, D, kTiles, kTwo>::kCtas)
    dense_tc_kernel(TcArgs p, Geom g, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap vrmap) {
    using C = CfgOf<T, D, kTiles, kTwo>;
    constexpr bool kBoth = kBothParts<T, kTwo>;
    constexpr int kEntriesK = kTwo ? 2 : 1, kEntriesV = kBoth ? 2 : 1;      // of the rings for a tile
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    using V = std::conditional_t<kTwo, __half, T>;
    constexpr bool kBf16V = std::is_same<V, __nv_bfloat16>::value;
    constexpr float kShift = kBf16V ? 0.f : 7.f;    // P is kept this much (log2) larger
    constexpr float kTop = kShift + 8.f;
    constexpr bool kOneK = kTwo && C::kStagesK == 1;      // K's two entries come one after the other in one place
    constexpr bool kDouble = kDoubleS<D, kMods> && !kOneK;
    constexpr int kPStep = kDouble || kBoth ? kHalf : kHalf / 2;      // TMEM columns from P's first half to its second
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* kt = smem + C::kKOff;
    uint8_t* vt = smem + C::kVOff;
    Ctl& c = *reinterpret_cast<Ctl*>(smem + C::kCtlOff);
    const DenseArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hkv;
    // units: key split fastest (the splits may be a cluster), then kv head (the heads of a cache row are neighbours), then
    // sequence, then the row tiles from the last one on (under the causal bound they see the most keys)
    int64_t u = blockIdx.x;
    const int split = (int)(u % a.splits);
    u /= a.splits;
    const int gkv = (int)(u % a.Hkv);
    u /= a.Hkv;
    const int b = (int)(u % g.B);
    const int tile = p.tiles - 1 - (int)(u / g.B);
    const int64_t m0 = (int64_t)tile * (kTiles * kRows);
    const int n_rows = (int)min((int64_t)g.T * G - m0, (int64_t)kTiles * kRows);   // packed rows of this CTA
    const int n_tiles = (n_rows + kRows - 1) / kRows;                              // row tiles with rows

    if (a.part_o) pdl_trigger();     // (the merge follows; results are not handed on early, see lidx_internal.cuh)
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&c.kfull[i], 1);
            mbar_init(&c.kempty[i], n_tiles);
            mbar_init(&c.vfull[i], 1);
            mbar_init(&c.vempty[i], n_tiles);
            mbar_init(&c.vok[i], 1);
        }
        for (int i = 0; i < n_tiles; ++i) {
            for (int x = 0; x < 2; ++x) {
                mbar_init(&c.sfull[i][x], 1);
                mbar_init(&c.pready[i][x], min(4, (n_rows - i * kRows + 31) / 32));   // warps with rows
            }
            mbar_init(&c.pvdone[i], 1);
            mbar_init(&c.odone[i], 1);
            mbar_init(&c.done[i], 1);
        }
        c.abort = 0;
        c.dirty = 0;
        c.k0 = INT32_MAX;
        c.k1 = 0;
        c.full0 = 0;
        c.full1 = INT32_MAX;
        fence_mbar_init();
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    if (warp == 0) {
        tmem_alloc(&c.tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    pdl_wait();
    __syncthreads();

    // ---- Q's rows on their way (they are stored below, after the other loads have been waited for)
    constexpr int kPieces = kTiles * C::kQRows * (D / 8), kPer = (kPieces + C::kThreads - 1) / C::kThreads;
    constexpr int kRowStep = C::kThreads / (D / 8);              // a thread's pieces: one column, rows this far apart
    const int t00 = (int)(m0 / G), h00 = (int)(m0 - (int64_t)t00 * G);   // token and head of the CTA's first row
    const int qr = threadIdx.x / (D / 8), qc = threadIdx.x % (D / 8);
    uint4 qv[kPer];
    {
        int t = (h00 + qr) / G, hh = (h00 + qr) - t * G;
        const int step_t = kRowStep / G, step_h = kRowStep - step_t * G;
        const T* q = static_cast<const T*>(a.q) + (((int64_t)b * g.T + t00) * a.Hq + gkv * G) * a.dk + qc * 8;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            qv[x] = make_uint4(0u, 0u, 0u, 0u);
            if (qr + x * kRowStep < n_rows && qc * 8 < a.dk)
                qv[x] = *reinterpret_cast<const uint4*>(q + ((int64_t)t * a.Hq + hh) * a.dk);
            t += step_t;
            hh += step_h;
            if (hh >= G) {
                hh -= G;
                ++t;
            }
        }
    }
    // ---- the rows: interval, position, slope; the CTA's keys
    const int n_kv = seq_n_kv(g, b);
    const int rt = (warp - kOtherWarps) >> 2;                       // this thread's row tile (softmax warps)
    const int r = (int)threadIdx.x - 32 * kOtherWarps;              // ... and row of the CTA
    const bool has_row = r >= 0 && r < n_rows;
    const bool warp_rows = warp >= kOtherWarps && r - lane < n_rows;  // some row of the warp is one
    Interval iv = {0, 0, 0};
    int64_t qrow = 0;
    int h = 0, wlo = 0, whi = INT32_MAX;    // keys that every row of the warp sees
    if (warp_rows) {
        if (has_row) {
            const int t = t00 + (h00 + r) / G;
            h = gkv * G + (h00 + r) % G;
            qrow = (int64_t)b * g.T + t;
            iv = row_interval(g, a.mods, qrow, b, n_kv);
        }
        const bool some = iv.lo < iv.hi;    // rows that see nothing take what they get and write zeros
        const int w0 = __reduce_min_sync(0xffffffffu, some ? iv.lo : INT32_MAX);
        const int w1 = __reduce_max_sync(0xffffffffu, some ? iv.hi : 0);
        wlo = __reduce_max_sync(0xffffffffu, some ? iv.lo : 0);
        whi = __reduce_min_sync(0xffffffffu, some ? iv.hi : INT32_MAX);
        if (lane == 0 && w1 > 0) {
            atomicMin(&c.k0, w0);
            atomicMax(&c.k1, w1);
            atomicMax(&c.full0, wlo);
            atomicMin(&c.full1, whi);
        }
    }
    // Q: 16-byte pieces into the swizzled K-major layout; rows and columns past the end are zero
    {
        uint8_t* qs = smem + (qc >> 3) * C::kQBlock;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int rr = qr + x * kRowStep, r0 = rr % C::kQRows;
            if (rr < kTiles * C::kQRows)
                *reinterpret_cast<uint4*>(qs + rr / C::kQRows * C::kQTile + r0 * 128 + (((qc & 7) ^ (r0 & 7)) << 4)) = qv[x];
        }
    }
    __syncthreads();
    // this split's keys: its share of the tiles (cuts of the position line) that some row of the CTA sees part of
    int k0 = c.k0, k1 = c.k1;
    const int64_t first = k0 / kKeys, tiles_seen = k1 > k0 ? (k1 + kKeys - 1) / kKeys - first : 0;
    // (where that is little of the line, as under a window, an equal share: 16 sequences of up to 32768 keys, window
    // 4096, 74 us in cuts of the line, 35 in equal shares; without a window 146 and 152: CTAs that end early leave
    // their SM's loads to the other there)
    const int64_t line = (g.max_n_kv + kKeys - 1) / kKeys;
    const int64_t share = ((2 * tiles_seen > line ? line : tiles_seen) + a.splits - 1) / a.splits;
    const int64_t s0 = (first + split * share) * kKeys, s1 = s0 + share * kKeys;
    if (k0 < s0) k0 = (int)(s0 < INT32_MAX ? s0 : INT32_MAX);
    if (k1 > s1) k1 = (int)s1;
    const int t0 = k0 / kKeys;
    const int n = k1 > k0 ? (k1 + kKeys - 1) / kKeys - t0 : 0;
    fence_proxy_async_smem();   // Q before the MMAs read it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem_base;
    const int full0 = c.full0, full1 = c.full1;

    if (n > 0) {
        auto aborted = [&] { return *(volatile int*)&c.abort != 0; };
        auto warp_aborted = [&] { return __any_sync(0xffffffffu, aborted()); };
        auto give_up = [&] {
            *(volatile int*)&c.abort = 1;
            flag(g.status, IDX_ERR_TIMEOUT);
        };
        if (warp == 0) {
            // -------------------------------------------------- producer: a lane per (piece, 64 columns)
            const int pieces = kKeys / p.box;
            const int64_t row_base = g.page_table ? 0 : seq_row0(g, b);
            int sent_k = 0, sent_v = 0;                // entries whose loads were issued
            auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int j) {
                if (lane == 0) mbar_arrive_expect_tx(bar, C::kTileBytes);
                __syncwarp();
                if (lane < pieces * (D / 64)) {
                    const int pc = lane / (D / 64), cb = lane % (D / 64);
                    const int64_t key = (int64_t)(t0 + j) * kKeys + pc * p.box;
                    // a piece that holds none of the keys is filled with zeros (a row past the cache), and so is
                    // one whose rows do not exist: the CTA's rows are redone key by key then
                    int64_t row = a.kv_rows;
                    if (key < k1 && key + p.box > k0) {
                        row = g.page_table ? key_row(g, b, key) : row_base + key;
                        if (row + max(k0 - key, (int64_t)0) < 0 || row + min(k1 - key, (int64_t)p.box) > a.kv_rows) {
                            row = a.kv_rows;
                            *(volatile int*)&c.dirty = 1;
                        }
                    }
                    tma_load_3d(dst + cb * kColBlock + pc * p.box * 128, map, bar, cb * 64, gkv, (int32_t)row);
                }
            };
            for (int j = 0; j < n; ++j) {
                bool ok = true;
#pragma unroll
                for (int x = 0; ok && x < kEntriesK; ++x) {
                    const int sk = sent_k % C::kStagesK;
                    ok = !warp_aborted() && warp_wait(&c.kempty[sk], (uint32_t)((sent_k / C::kStagesK) & 1) ^ 1);
                    if (!ok) break;
                    load(x ? &rmap : &kmap, kt + sk * C::kTileBytes, &c.kfull[sk], j);
                    ++sent_k;
                }
#pragma unroll
                for (int x = 0; ok && x < kEntriesV; ++x) {
                    const int sv = sent_v % C::kStagesV;
                    ok = !warp_aborted() && warp_wait(&c.vempty[sv], (uint32_t)((sent_v / C::kStagesV) & 1) ^ 1);
                    if (!ok) break;
                    load(x ? &vrmap : &vmap, vt + sv * C::kTileBytes, &c.vfull[sv], j);
                    ++sent_v;
                }
                if (!ok) {
                    give_up();
                    break;
                }
            }
            if (warp_aborted()) {
                // no load may still be in flight when the CTA ends
                for (int j = max(0, sent_k - C::kStagesK); j < sent_k; ++j)
                    warp_wait(&c.kfull[j % C::kStagesK], (uint32_t)((j / C::kStagesK) & 1));
                for (int j = max(0, sent_v - C::kStagesV); j < sent_v; ++j)
                    warp_wait(&c.vfull[j % C::kStagesV], (uint32_t)((j / C::kStagesV) & 1));
            }
        } else if (warp <= n_tiles) {
            // -------------------------------------------------- MMA issuers, one warp per row tile.  The warp walks
            // together and a lane issues: operands that all lanes share stay in uniform registers (with one lane on
            // its own a product took about 100 cycles to issue, more than it takes).  The queue of issued products is
            // short, so the tensor pipe idles while an issuer waits or commits: it has the other issuer's then.
            const int i = warp - 1;
            const uint32_t id_qk = idesc_f16_f32_major(kRows, kDouble ? kHalf : kKeys, kBf16 ? 1 : 0, 0, 0);
            const uint32_t id_pv = idesc_f16_f32_major(kRows, (a.dv + 15) & ~15, kBf16V ? 1 : 0, 0, 1);
            const uint64_t kmajor = desc_sw128_kmajor(0, 1024), mnmajor = desc_sw128_mnmajor(0, kColBlock, 1024);
            const uint32_t k_hi = desc_hi(kmajor), v_hi = desc_hi(mnmajor), k_lo = (uint32_t)kmajor, v_lo = (uint32_t)mnmajor;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t qa = __shfl_sync(0xffffffffu, k_lo + desc_addr(smem) + (i * C::kQTile >> 4), 0);
            const uint32_t kb = k_lo + desc_addr(kt), vb = v_lo + desc_addr(vt);
            const uint32_t ts = __shfl_sync(0xffffffffu, tm + i * kKeys, 0);
            const uint32_t to = __shfl_sync(0xffffffffu, tm + C::kOCol + i * D, 0);
            int sk = 0, kph = 0, sv = 0, vph = 0;     // ring positions of the K tile and the V tile to use next
            bool ok = true;
            // S = Q K^T.  All D / 16 products run (columns past dk are zero): an unrolled chain that stopped at dk by
            // a run-time bound got a wrong last descriptor (nvcc 13.0; the basis-vector test shows it)
            auto qk = [&](int half) {
                const int s2 = kTwo ? (sk + 1 == C::kStagesK ? 0 : sk + 1) : sk;      // the second entry
                const uint32_t ka = __shfl_sync(0xffffffffu, kb + ((sk * C::kTileBytes + half * (kHalf * 128)) >> 4), 0);
                const uint32_t kr = __shfl_sync(0xffffffffu, kb + ((s2 * C::kTileBytes + half * (kHalf * 128)) >> 4), 0);
                const uint32_t d = __shfl_sync(0xffffffffu, ts + half * kHalf, 0);
                const bool last = !kDouble || half == 1;      // of the K tile
                tc_fence_after();
                auto product = [&](uint32_t k, uint32_t add) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_f16_ss_lo(d, qa + (((ks >> 2) * C::kQBlock + (ks & 3) * 32) >> 4), k_hi,
                                      k + (((ks >> 2) * kColBlock + (ks & 3) * 32) >> 4), k_hi, id_qk, ks > 0 ? 1u : add);
                };
                bool there = true;
                if constexpr (kOneK) {
                    if (elect_one()) {
                        product(ka, 0u);
                        mma_commit(&c.kempty[0]);
                    }
                    __syncwarp();
                    there = warp_wait(&c.kfull[0], (uint32_t)kph ^ 1);
                    tc_fence_after();
                }
                if (elect_one()) {
                    if (!kOneK) product(ka, 0u);
                    if constexpr (kTwo) {
                        if (!kOneK && last) mma_commit(&c.kempty[sk]);
                        if (there) product(kr, 1u);
                    }
                    mma_commit(&c.sfull[i][half]);
                    if (last) mma_commit(&c.kempty[s2]);
                }
                __syncwarp();
                if (last)
                    for (int x = 0; x < (kTwo ? 2 : 1); ++x)
                        if (++sk == C::kStagesK) {
                            sk = 0;
                            kph ^= 1;
                        }
                return there;
            };
            // the K tile to use next is there
            auto wait_k = [&] {
                bool there = warp_wait(&c.kfull[sk], (uint32_t)kph);
                if (kTwo && !kOneK)
                    there = there && (sk + 1 == C::kStagesK ? warp_wait(&c.kfull[0], (uint32_t)kph ^ 1)
                                                            : warp_wait(&c.kfull[sk + 1], (uint32_t)kph));
                return there;
            };
            // O += P V of half a tile, and the commits that follow it
            auto second_v = [&] { return kBoth ? (sv + 1 == C::kStagesV ? 0 : sv + 1) : sv; };      // the second entry
            auto pv = [&](int half, uint32_t first, uint64_t* b0, uint64_t* b1, uint64_t* b2) {
                const uint32_t va = __shfl_sync(0xffffffffu, vb + ((sv * C::kTileBytes + half * (kHalf * 128)) >> 4), 0);
                const uint32_t vr = __shfl_sync(0xffffffffu, vb + ((second_v() * C::kTileBytes + half * (kHalf * 128)) >> 4), 0);
                const uint32_t pa = __shfl_sync(0xffffffffu, ts + half * kPStep, 0);
                const uint32_t acc = __shfl_sync(0xffffffffu, first ? 0u : 1u, 0);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kHalf / 16; ++ks)
                        mma_f16_ts_lo(to, pa + ks * 8, va + (ks * 2048 >> 4), v_hi, id_pv, ks > 0 ? 1u : acc);
                    if constexpr (kBoth) {
#pragma unroll
                        for (int ks = 0; ks < kHalf / 16; ++ks)
                            mma_f16_ts_lo(to, pa + kHalf / 2 + ks * 8, va + (ks * 2048 >> 4), v_hi, id_pv, 1u);
#pragma unroll
                        for (int ks = 0; ks < kHalf / 16; ++ks)
                            mma_f16_ts_lo(to, pa + ks * 8, vr + (ks * 2048 >> 4), v_hi, id_pv, 1u);
                    }
                    if (b0) mma_commit(b0);
                    if (b1) mma_commit(b1);
                    if (b2) mma_commit(b2);
                }
                __syncwarp();
            };
            ok = wait_k();
            if (ok) ok = qk(0);
            if (ok && kDouble) ok = qk(1);
            for (int j = 0; ok && j < n; ++j) {
                const bool last = j + 1 == n;
                ok = warp_wait(&c.vok[sv], (uint32_t)vph) &&
                     (!kBoth || warp_wait(&c.vok[second_v()], (uint32_t)(second_v() > sv ? vph : vph ^ 1))) &&
                     warp_wait(&c.pready[i][0], (uint32_t)(j & 1));
                if (!ok) break;
                // new scores follow the product over the weights that they replace: a row tile's products run in order.
                // (Two buffers: the commit after the last tile's first half has no scores; it tells that the products
                // of the step before are complete, as scores would.)
                if (kDouble) {
                    pv(0, j == 0, last ? &c.sfull[i][0] : nullptr, nullptr, nullptr);
                    if (!last) {
                        ok = wait_k();
                        if (!ok) break;
                        ok = qk(0);
                    }
                } else {
                    pv(0, j == 0, &c.pvdone[i], nullptr, nullptr);
                    ok = last || wait_k();
                }
                ok = ok && warp_wait(&c.pready[i][1], (uint32_t)(j & 1));
                if (!ok) break;
                pv(1, false, &c.vempty[sv], last ? &c.odone[i] : nullptr, kBoth ? &c.vempty[second_v()] : nullptr);
                if (!last) ok = qk(kDouble ? 1 : 0);
                for (int x = 0; x < kEntriesV; ++x)
                    if (++sv == C::kStagesV) {
                        sv = 0;
                        vph ^= 1;
                    }
            }
            if (!ok) give_up();
            if (elect_one()) mma_commit(&c.done[i]);
            __syncwarp();
            warp_wait(&c.done[i], 0);
        } else if (warp == kOtherWarps - 1) {
            // -------------------------------------------------- V inspector: tiles that some row sees in part
            for (int x = 0; x < n * kEntriesV; ++x) {
                const int sv = x % C::kStagesV;
                if (warp_aborted() || !warp_wait(&c.vfull[sv], (uint32_t)((x / C::kStagesV) & 1))) {
                    give_up();
                    break;
                }
                const int key0 = (t0 + x / kEntriesV) * kKeys;
                if (key0 < max(full0, k0) || key0 + kKeys > min(full1, k1)) {
                    uint8_t* v = vt + sv * C::kTileBytes;
                    bool found = false;
                    // four lanes per V row and column block (rows of 128 bytes)
                    for (int e = lane; e < kKeys * 4 * (D / 64); e += 32) {
                        const int row = (e >> 2) & (kKeys - 1), cb = e / (kKeys * 4);
                        uint4* at = reinterpret_cast<uint4*>(v + cb * kColBlock + row * 128 + (e & 3) * 32);
                        if (key0 + row < k0 || key0 + row >= k1) {
                            at[0] = at[1] = make_uint4(0u, 0u, 0u, 0u);
                        } else if (key0 + row < full0 || key0 + row >= full1) {
                            const uint4 y[2] = {at[0], at[1]};
                            const uint32_t* z = reinterpret_cast<const uint32_t*>(y);
                            constexpr uint32_t kExp = kBf16V ? 0x7F80u : 0x7C00u;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                found |= (z[i] & kExp) == kExp || (z[i] & (kExp << 16)) == (kExp << 16);
                        }
                    }
                    if (__any_sync(0xffffffffu, found) && lane == 0) *(volatile int*)&c.dirty = 1;
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.vok[sv]);
            }
        }
    }
    // -------------------------------------------------------------- softmax and output (thread = row)
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lane_off + C::kOCol + rt * D;
    const bool merge = a.splits > 1 && !a.part_o;     // the splits are the CTAs of a cluster
    float m_used = -INFINITY, l_run = 0.f;
    bool ok = n > 0;
    if (warp_rows) {
        const uint32_t ts = tmem + lane_off + rt * kKeys;
        const Score sc = [&] {
            const float slope = a.mods.slopes && has_row ? a.mods.slopes[h] : 0.f;
            if constexpr (kBoth) {
                // (from one lane, for all: a uniform register)
                const float scale = a.scale * exp2_whole(k_exponent(a.v_top[(int64_t)(g.B + b) * a.Hkv + gkv]));
                return make_score(a, __shfl_sync(0xffffffffu, kMods ? scale : fmaxf(scale, 0x1p-126f), 0), slope);      // (still above 0)
            } else {
                return make_score(a, a.scale, slope);
            }
        }();
        auto timed_out = [&] {
            *(volatile int*)&c.abort = 1;
            flag(g.status, IDX_ERR_TIMEOUT);
            ok = false;
        };
        const uint64_t c2 = pair(sc.c, sc.c);
        // the warp's rows see nothing past their own positions; its first position
        const bool past = __all_sync(0xffffffffu, iv.hi <= iv.pos + 1 || iv.lo >= iv.hi);
        const int first_pos = __reduce_min_sync(0xffffffffu, iv.lo < iv.hi ? iv.pos : INT32_MAX);
        for (int q = 0; ok && q < 2 * n; ++q) {
            const int j = q >> 1, half = q & 1;
            if (kDouble || half == 0) {
                if (!warp_wait(&c.sfull[rt][kDouble ? half : 0], (uint32_t)(j & 1))) {
                    timed_out();
                    break;
                }
                tc_fence_after();
            }
            const int key0 = (t0 + j) * kKeys + half * kHalf;
            float s[kHalf];
            {
                uint32_t x[32], y[32];
                tmem_ld_32x32b_x32_raw(ts + half * kHalf, x);
                tmem_ld_32x32b_x32_raw(ts + half * kHalf + 32, y);
                tmem_ld_wait_for(x);
                tmem_ld_wait_for(y);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    s[i] = __uint_as_float(x[i]);
                    s[32 + i] = __uint_as_float(y[i]);
                }
            }
            if (kMods) modify(s, sc, (float)(iv.pos - key0), past || key0 + kHalf <= first_pos);
            if (key0 < wlo || key0 < k0 || key0 + kHalf > whi || key0 + kHalf > k1) {
                // visible columns [a0, a1) of this row, as bits
                const int a0 = min(max(max(iv.lo, k0) - key0, 0), kHalf), a1 = max(min(min(iv.hi, k1) - key0, kHalf), 0);
                const uint64_t up = a0 >= kHalf ? 0ull : ~0ull << a0, down = a1 >= kHalf ? ~0ull : (1ull << a1) - 1ull;
                const uint32_t m0 = (uint32_t)(up & down), m1 = (uint32_t)((up & down) >> 32);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    s[i] = (m0 >> i) & 1u ? s[i] : -INFINITY;
                    s[32 + i] = (m1 >> i) & 1u ? s[32 + i] : -INFINITY;
                }
            }
            // the row's maximum
            float x0 = fmaxf(s[0], s[1]), x1 = fmaxf(s[2], s[3]), x2 = fmaxf(s[4], s[5]), x3 = fmaxf(s[6], s[7]);
#pragma unroll
            for (int i = 8; i < kHalf; i += 8) {
                x0 = fmaxf(fmaxf(x0, s[i]), s[i + 1]);
                x1 = fmaxf(fmaxf(x1, s[i + 2]), s[i + 3]);
                x2 = fmaxf(fmaxf(x2, s[i + 4]), s[i + 5]);
                x3 = fmaxf(fmaxf(x3, s[i + 6]), s[i + 7]);
            }
            float mt = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
            if (!kMods) mt *= sc.c;     // c > 0 here: the largest product gives the largest score
            const bool rise = mt > m_used + kTop || (m_used == -INFINITY && mt > -INFINITY);
            if (__any_sync(0xffffffffu, rise)) {
                float al = 1.f;
                if (rise) {
                    const float to_m = mt - kShift;
                    al = m_used == -INFINITY ? 1.f : ex2_approx(m_used - to_m);
                    m_used = to_m;
                    l_run *= al;
                }
                if (q > 0 && __any_sync(0xffffffffu, al != 1.f)) {
                    // O's products up to here.  One buffer: those of the tile before are complete (this S came after
                    // them), the first half's of this one has to be waited for.  Two: the next step's scores came
                    // after the last step's product.
                    if (kDouble ? !warp_wait(&c.sfull[rt][half ^ 1], (uint32_t)(((q + 1) >> 1) & 1))
                                : half == 1 && !warp_wait(&c.pvdone[rt], (uint32_t)(j & 1))) {
                        timed_out();
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int cb = 0; cb < D / 32; ++cb) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32_raw(to + cb * 32, o);
                        tmem_ld_wait_for(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                        tmem_st_32x32b_x32(to + cb * 32, o);
                    }
                }
            }
            const float nm = m_used == -INFINITY ? 0.f : -m_used;
            const uint64_t nm2 = pair(nm, nm);
            uint64_t la = 0ull, lb = 0ull;
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < kHalf; i += 2) {
                const uint64_t e = kMods ? add2(pair(s[i], s[i + 1]), nm2) : fma2(pair(s[i], s[i + 1]), c2, nm2);
                float p0, p1;
                unpair(e, p0, p1);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                if (i & 2)
                    la = add2(la, pair(p0, p1));
                else
                    lb = add2(lb, pair(p0, p1));
                w[i / 2] = pack2<V>(p0, p1);
                if constexpr (kBoth) {
                    s[i] = p0;
                    s[i + 1] = p1;
                }
            }
            tmem_st_32x32b_x32(ts + half * kPStep, w);
            if constexpr (kBoth) {      // what the rounding took off
#pragma unroll
                for (int i = 0; i < kHalf; i += 2) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
                    w[i / 2] = pack2<V>(s[i] - x.x, s[i + 1] - x.y);
                }
                tmem_st_32x32b_x32(ts + half * kPStep + kHalf / 2, w);
            }
            float l0, l1;
            unpair(add2(la, lb), l0, l1);
            l_run += l0 + l1;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.pready[rt][half]);
        }
        if (ok) ok = warp_wait(&c.odone[rt], 0);
        tc_fence_after();
    }
    // merged in the cluster, the rows' unnormalised results are kept over all of the ring
    if (merge) __syncthreads();
    if (warp_rows) {
        const bool some = iv.lo < iv.hi;
        const int64_t rh = qrow * a.Hq + h;
        // every tile has been loaded and looked over by now: each PV product waited for that
        const bool by_key = ok && *(volatile int*)&c.dirty != 0;
        float acc[D];
        if (by_key) {
            float ml[2] = {-INFINITY, 0.f};
            if (has_row && some) scalar_row<T, V>(a, g, b, gkv, rh, h, iv, s0, s1, acc, ml);
            m_used = ml[0];
            l_run = ml[1];
            __syncwarp();
        }
        const float l = some && ok ? l_run : 0.f;
        const float unit = kTwo ? exp2_whole(v_exponent(a.v_top[(int64_t)b * a.Hkv + gkv])) : 1.f;
        const float inv = l == 0.f ? 0.f : a.splits > 1 ? unit : unit / l;
        if (merge) {
            *reinterpret_cast<float2*>(smem + C::kMlOff + r * 8) = make_float2(m_used, l);
        } else if (has_row) {
            if (a.splits > 1) {
                a.part_ml[(rh * a.splits + split) * 2] = m_used * kLn2;
                a.part_ml[(rh * a.splits + split) * 2 + 1] = l;
            } else if (a.lse) {
                a.lse[rh] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * kLn2;
            }
        }
        // through shared memory (Q's, and past it K's: no product reads them any more), so that whole rows are written;
        // normalised (a split's partial: as they are)
        uint8_t* rows = merge ? smem + (rt * kRows + (warp & 3) * 32) * (D * 4) : smem + rt * C::kQTile + (warp & 3) * (32 * D * 2);
        const bool parts = a.splits > 1;
        const int W = merge || !parts ? D : D / 2;
#pragma unroll 1
        for (int c0 = 0; c0 < a.dv; c0 += W) {
#pragma unroll 1
            for (int x = 0; x < W; x += 32) {
                uint32_t u32[32];
                float o[32];
                if (by_key) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) u32[i] = __float_as_uint(acc[c0 + x + i]);
                } else if (ok) {
                    tmem_ld_32x32b_x32_raw(to + c0 + x, u32);
                    tmem_ld_wait_for(u32);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : __uint_as_float(u32[i]) * inv;
                if (merge)
                    stage_cols<float, D>(rows, lane, x, o);
                else if (parts)
                    stage_cols<float, D / 2>(rows, lane, x, o);
                else
                    stage_cols<T, D>(rows, lane, x, o);
            }
            if (merge) break;
            if (parts)
                store_rows<float, D / 2>(a.part_o + c0, (rh * a.splits + split) * a.dv, n_rows - (r - lane), rows,
                                         min(W, a.dv - c0));
            else
                store_rows<T, D>(static_cast<T*>(a.out), rh * a.dv, n_rows - (r - lane), rows, a.dv);
        }
        tc_fence_before();
    }
    if (merge) {
        // ---------------------------------------------------------- the splits' results: each CTA merges its share of
        // the rows' 8-column pieces, in the order of the splits
        cluster_sync();
        const int pieces = a.dv / 8;
        for (int e = split * C::kThreads + threadIdx.x; e < n_rows * pieces; e += a.splits * C::kThreads) {
            const int row = e / pieces, pc = e - row * pieces;
            float M = -INFINITY;
            for (int s = 0; s < a.splits; ++s) {
                const float2 ml = *reinterpret_cast<const float2*>(of_cta(smem + C::kMlOff + row * 8, s));
                if (ml.y != 0.f) M = fmaxf(M, ml.x);
            }
            float den = 0.f, o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = 0.f;
            for (int s = 0; s < a.splits; ++s) {
                const float2 ml = *reinterpret_cast<const float2*>(of_cta(smem + C::kMlOff + row * 8, s));
                if (ml.y == 0.f) continue;
                const float w = exp2f(ml.x - M);
                den = fmaf(w, ml.y, den);
                const uint8_t* x = of_cta(smem + row * (D * 4), s);
                const float4 x0 = *reinterpret_cast<const float4*>(x + (((2 * pc) ^ (row & 7)) << 4));
                const float4 x1 = *reinterpret_cast<const float4*>(x + (((2 * pc + 1) ^ (row & 7)) << 4));
                o[0] = fmaf(w, x0.x, o[0]);
                o[1] = fmaf(w, x0.y, o[1]);
                o[2] = fmaf(w, x0.z, o[2]);
                o[3] = fmaf(w, x0.w, o[3]);
                o[4] = fmaf(w, x1.x, o[4]);
                o[5] = fmaf(w, x1.y, o[5]);
                o[6] = fmaf(w, x1.z, o[6]);
                o[7] = fmaf(w, x1.w, o[7]);
            }
            const float inv = den == 0.f ? 0.f : 1.f / den;
            const int64_t rh = ((int64_t)b * g.T + t00 + (h00 + row) / G) * a.Hq + gkv * G + (h00 + row) % G;
            if (a.lse && pc == 0) a.lse[rh] = den == 0.f ? -INFINITY : (M + log2f(den)) * kLn2;
            *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + rh * a.dv + pc * 8) =
                make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                           pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
        }
        cluster_sync();     // no CTA leaves while another reads its memory
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, C::kTmemCols);
}

// row tiles per CTA
int row_tiles(int64_t packed) { return packed > kFewRows ? 2 : 1; }

template <typename T, int D, int kTiles, bool kMods, bool kTwo>
cudaError_t go(const TcArgs& p, const Geom& g, const CUtensorMap* m, int64_t grid, cudaStream_t st) {
    using C = CfgOf<T, D, kTiles, kTwo>;
    constexpr size_t sm = 1024 + (size_t)C::kCtlOff + sizeof(Ctl);
    static_assert((sm + 1024) * C::kCtas <= 233472, "shared memory of an SM");
    auto kern = dense_tc_kernel<T, D, kTiles, kMods, kTwo>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kern, dim3((unsigned)grid), dim3(C::kThreads), sm, st,
                              p.a.splits > 1 && !p.a.part_o ? p.a.splits : 1, p, g, m[0], m[1], m[2], m[3]);
}

template <typename T, bool kTwo>
cudaError_t run(const DenseArgs& a, const Geom& g, cudaStream_t st) {
    const int64_t packed = (int64_t)g.T * (a.Hq / a.Hkv);
    const int tiles = row_tiles(packed);
    TcArgs p = {a, (int)((packed + tiles * kRows - 1) / (tiles * kRows)), box_rows(g.page_size, kKeys)};
    const int64_t grid = (int64_t)g.B * a.Hkv * p.tiles * a.splits;
    if (grid > INT32_MAX) return cudaErrorNotSupported;
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    CUtensorMap m[4];      // K, V, and what they lack
    if (!make_head_tmap(&m[0], a.k, bf16, a.dk, a.Hkv, a.k_stride, a.kv_rows, p.box) ||
        !make_head_tmap(&m[1], a.v, bf16 && !kTwo, a.dv, a.Hkv, a.v_stride, a.kv_rows, p.box))
        return cudaErrorNotSupported;
    m[2] = m[0];
    m[3] = m[1];
    if (kTwo && !make_head_tmap(&m[2], a.k_rest, bf16, a.dk, a.Hkv, a.k_stride, a.kv_rows, p.box)) return cudaErrorNotSupported;
    if (kBothParts<T, kTwo> && !make_head_tmap(&m[3], a.v_rest, false, a.dv, a.Hkv, a.v_stride, a.kv_rows, p.box))
        return cudaErrorNotSupported;
    const bool small = a.dk <= 64 && a.dv <= 64;
    const bool mods = a.mods.softcap > 0.f || a.mods.slopes || a.scale <= 0.f;
    if (small) {
        if (tiles == 1)
            return mods ? go<T, 64, 1, true, kTwo>(p, g, m, grid, st) : go<T, 64, 1, false, kTwo>(p, g, m, grid, st);
        return mods ? go<T, 64, 2, true, kTwo>(p, g, m, grid, st) : go<T, 64, 2, false, kTwo>(p, g, m, grid, st);
    }
    if (tiles == 1)
        return mods ? go<T, 128, 1, true, kTwo>(p, g, m, grid, st) : go<T, 128, 1, false, kTwo>(p, g, m, grid, st);
    return mods ? go<T, 128, 2, true, kTwo>(p, g, m, grid, st) : go<T, 128, 2, false, kTwo>(p, g, m, grid, st);
}

}  // namespace

bool dense_tc_supported(const DenseArgs& a, int dtype, const Geom& g) {
    if (dtype == IDX_F32 || !a.v || a.dk > 128 || a.dv > 128 || a.dk % 8 || a.dv % 8) return false;
    if (a.kv_rows < 1 || a.kv_rows > INT32_MAX - kKeys || a.k_stride % 8 || a.v_stride % 8) return false;
    // pages are loaded in boxes of whole 8-row swizzle groups
    if (g.page_table && box_rows(g.page_size, kKeys) < 8) return false;
    const uint64_t all = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                         reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.out);
    return all % 16 == 0;
}

// as many splits as keep the CTAs within twice the SMs (one round for calls of few rows, with two CTAs to an SM), and no
// more than there are pieces of 512 keys; 513 keys are two pieces
int dense_tc_splits(int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv) {
    const int64_t packed = n_q * (Hq / Hkv);
    const int64_t rows = row_tiles(packed) * kRows;
    const int64_t units = n_seq * Hkv * ((packed + rows - 1) / rows);
    int sms = sm_count();
    if (sms < 2) sms = 152;
    if (units < 1) return 1;
    int64_t s = 2 * (int64_t)sms / units;
    const int64_t by_keys = (max_n_kv + 511) / 512;
    if (s > by_keys) s = by_keys;
    if (s > kDenseMaxSplits) s = kDenseMaxSplits;
    return s < 1 ? 1 : (int)s;
}

cudaError_t launch_dense_tc(const DenseArgs& a, int dtype, const Geom& g, cudaStream_t st) {
    if (a.k_rest) return dtype == IDX_BF16 ? run<__nv_bfloat16, true>(a, g, st) : run<__half, true>(a, g, st);
    return dtype == IDX_BF16 ? run<__nv_bfloat16, false>(a, g, st) : run<__half, false>(a, g, st);
}

}  // namespace lidx
