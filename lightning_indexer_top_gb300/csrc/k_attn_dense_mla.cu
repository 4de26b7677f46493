// Dense attention over a (paged) MLA latent cache on the tensor cores: 128 query
// heads, bf16 rows of 576 columns, value = the first 512 (dense_attn in lidx.h).
//
// The unit is that of the sparse MLA attention (attn_mla_tc.cuh: a 2-CTA cluster
// per query row and key split, rank 0 scores and softmax, rank 1 the values), fed
// with whole runs of the position line instead of a selection: the key tiles are
// 64 consecutive positions, loaded by TMA boxes of at most a page (the sparse
// unit's 16-byte gathers reach about 36 GB/s per SM; a 72 KB tile takes 2 us).
// Every head of a query row sees the same keys, so a tile needs one bit per key;
// rows without their bit (a page's unwritten end, a page out of range) are zeroed
// in rank 1's tile before it is multiplied, so that nothing in them reaches the
// output.  Splits are merged by a kernel of their own, which also writes lse.
#include "attn_mla_tc.cuh"
#include "dense_attn.cuh"

namespace lidx {
namespace {
using namespace sm100;

struct DenseParams {
    DenseArgs a;
    int box;          // rows per TMA box: 64, or the largest power of two that divides the page
    int kps;          // keys of the position line per split
};

template <bool kScoreMods>
struct DenseFeed {
    static constexpr bool kDense = true;
    static constexpr bool kMods = kScoreMods;
    const CUtensorMap* map;
    const DenseParams* p;
    int base;         // position of the unit's first tile
    int pos;          // the query row's position

    // one warp: tile t's column blocks, a lane per (piece of the tile, block)
    template <int kBlocks, int kNStages, int kStageBytes>
    __device__ __forceinline__ void load_tiles(Ctl& c, uint8_t* xtiles, const Unit& u, const uint32_t* vmask, int producer,
                                               const Geom& g) const {
        if (producer != 0) return;
        const int lane = threadIdx.x & 31;
        const int pieces = kKeys / p->box;
        int sent = 0;
        fence_proxy_async_smem();    // what was read or written here before (Q's staging) is done with
        for (int t = 0; t < u.n_tiles; ++t) {
            const int stage = t % kNStages;
            if (warp_aborted(c) || !warp_wait(&c.xempty[stage], (uint32_t)((t / kNStages) & 1) ^ 1)) {
                abort_cta(c, g.status);
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&c.xfull[stage], kBlocks * kBlockBytes);
            __syncwarp();
            const uint64_t seen = (uint64_t)vmask[2 * t] | (uint64_t)vmask[2 * t + 1] << 32;
            for (int e = lane; e < pieces * kBlocks; e += 32) {
                const int pc = e / kBlocks, cb = e - pc * kBlocks;
                const uint64_t bits = p->box == 64 ? ~0ull : ((1ull << p->box) - 1ull) << (pc * p->box);
                // a piece without a key to see is filled with zeros (a row past the cache)
                int64_t row = p->a.kv_rows;
                if (seen & bits) row = key_row(g, u.b, (int64_t)base + t * kKeys + pc * p->box);
                tma_load_3d(xtiles + (size_t)stage * kStageBytes + cb * kBlockBytes + pc * p->box * 128, map,
                            &c.xfull[stage], cb * 64, 0, (int32_t)row);
            }
            sent = t + 1;
        }
        if (warp_aborted(c))    // no load may still be in flight when the CTA ends
            for (int t = max(0, sent - kNStages); t < sent; ++t)
                warp_wait(&c.xfull[t % kNStages], (uint32_t)((t / kNStages) & 1));
    }

    // one warp of rank 1: zero the value rows that are not seen
    __device__ __forceinline__ void zero_unseen(Ctl& c, uint8_t* xtiles, const Unit& u, const uint32_t* vmask,
                                                const Geom& g) const {
        const int lane = threadIdx.x & 31;
        for (int t = 0; t < u.n_tiles; ++t) {
            const int stage = t % kStagesV;
            if (warp_aborted(c) || !warp_wait(&c.xfull[stage], (uint32_t)((t / kStagesV) & 1))) {
                abort_cta(c, g.status);
                break;
            }
            const uint64_t seen = (uint64_t)vmask[2 * t] | (uint64_t)vmask[2 * t + 1] << 32;
            if (seen != ~0ull) {
                for (int e = lane; e < kKeys * kDvBlocks * 8; e += 32) {
                    const int row = (e >> 3) & (kKeys - 1), cb = e / (kKeys * 8);
                    if (!((seen >> row) & 1ull))
                        *reinterpret_cast<uint4*>(xtiles + (size_t)stage * kVTileBytes + cb * kBlockBytes + row * 128 +
                                                  (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&c.vok[stage]);
        }
    }

    __device__ __forceinline__ void modify(float (&s0)[32], float (&s1)[32], const Unit& u, int t, int h) const {
        (void)u;
        const Score sc = make_score(p->a, p->a.mods.slopes ? p->a.mods.slopes[h] : 0.f);
        const float d = (float)(pos - (base + t * kKeys));
        const bool past = base + (t + 1) * kKeys <= pos + 1;      // (every head of the row alike)
        lidx::modify(s0, sc, d, past);
        lidx::modify(s1, sc, d - 32.f, past);
    }

    __device__ __forceinline__ void store_lse(int64_t rh, float m, float l) const {
        if (p->a.lse) p->a.lse[rh] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
};

// every warp but the Q loaders: one bit per key of the unit's tiles
__device__ __forceinline__ void stage_bits(const MlaSmem& sm, uint32_t rank, const Unit& u, const Geom& g, int base,
                                           int lo, int hi, int64_t kv_rows) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_st = rank == 0 ? kThreads / 32 - 4 : kThreads / 32;
    const int si = rank == 0 && warp > 5 ? warp - 4 : warp;
    for (int w = si; w < u.n_tiles * (kKeys / 32); w += n_st) {
        const int j = base + w * 32 + lane;
        bool seen = j >= lo && j < hi;
        if (seen) {
            const int64_t row = key_row(g, u.b, j);
            if (row < 0 || row >= kv_rows) {
                seen = false;
                if (rank == 0) flag(g.status, IDX_ERR_DEVICE_BOUNDS);
            }
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, seen);
        if (lane == 0) sm.vmask[w] = bits;
    }
}

template <bool kScoreMods>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_mla_kernel(DenseParams p, Geom g, int64_t n_units, const __grid_constant__ CUtensorMap map) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const MlaSmem sm = mla_smem(smem);
    Ctl& c = *sm.c;
    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x >> 5;
    const int64_t n_clusters = gridDim.x >> 1;
    const DenseArgs& a = p.a;
    if (a.part_o) pdl_trigger();     // (the merge follows; results are not handed on early, see lidx_internal.cuh)
    if (threadIdx.x == 0) {
        mla_init(c, 1);
        tma_prefetch_desc(&map);
    }
    if (warp == 1) {
        tmem_alloc(&c.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem_base;
    pdl_wait();
    for (int64_t unit = blockIdx.x >> 1; unit < n_units; unit += n_clusters) {
        if (unit != (int64_t)(blockIdx.x >> 1)) {
            if (threadIdx.x == 0) mla_init(c, 1);
            __syncthreads();
        }
        Unit u;
        u.r = unit / a.splits;
        const int split = (int)(unit % a.splits);
        u.b = (int)(u.r / g.T);
        u.n_kv = seq_n_kv(g, u.b);
        u.fallback = 0;
        const Interval iv = row_interval(g, a.mods, u.r, u.b, u.n_kv);
        const int64_t s0 = (int64_t)split * p.kps;
        const int lo = (int)max((int64_t)iv.lo, s0), hi = (int)min((int64_t)iv.hi, s0 + p.kps);
        const int base = lo / kKeys * kKeys;      // tiles are cuts of the position line
        u.k0 = lo;
        u.k1 = hi;
        u.n_tiles = hi > lo ? (hi - base + kKeys - 1) / kKeys : 0;
        const bool q_warp = mla_q_warp(rank);
        if (q_warp) mla_load_q(c, sm.xtiles, tmem, static_cast<const __nv_bfloat16*>(a.q), u.r);
        else stage_bits(sm, rank, u, g, base, lo, hi, a.kv_rows);
        tc_fence_before();
        cluster_sync();
        tc_fence_after();
        const DenseFeed<kScoreMods> feed = {&map, &p, base, iv.pos};
        mla_run(sm, tmem, rank, u, unit, static_cast<const __nv_bfloat16*>(a.k), a.k_stride, g, a.scale * kLog2e, a.splits,
                a.out, IDX_BF16, a.part_o, a.part_ml, feed);
        tc_fence_before();
        __syncthreads();
        cluster_sync();
        tc_fence_after();
    }
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, block (row, kCols columns), thread = head
constexpr int kCols = 8;
__global__ void __launch_bounds__(kHq) dense_mla_combine_kernel(DenseArgs a) {
    pdl_wait();
    const int64_t r = blockIdx.x;
    const int h = threadIdx.x;
    // the splits' loads kBatch at a time
    constexpr int kBatch = 8;
    float M = -INFINITY;
    for (int s0 = 0; s0 < a.splits; s0 += kBatch) {
        float2 ml[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            ml[k] = s0 + k < a.splits ? reinterpret_cast<const float2*>(a.part_ml)[(r * a.splits + s0 + k) * kHq + h]
                                      : make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (ml[k].y != 0.f) M = fmaxf(M, ml[k].x);
    }
    float acc[kCols], den = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
    for (int s0 = 0; s0 < a.splits; s0 += kBatch) {
        float2 ml[kBatch];
        float4 x[kBatch][kCols / 4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t u = r * a.splits + min(s0 + k, a.splits - 1);
            ml[k] = reinterpret_cast<const float2*>(a.part_ml)[u * kHq + h];
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i)
                x[k][i] = reinterpret_cast<const float4*>(a.part_o + u * (int64_t)kDv * kHq)[(int64_t)(blockIdx.y * (kCols / 4) + i) * kHq + h];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const bool in = s0 + k < a.splits && ml[k].y != 0.f;
            const float w = in ? exp2f(ml[k].x - M) : 0.f;
            den += in ? w * ml[k].y : 0.f;
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i) {
                // (a split without keys wrote zeros)
                acc[4 * i] = fmaf(w, x[k][i].x, acc[4 * i]);
                acc[4 * i + 1] = fmaf(w, x[k][i].y, acc[4 * i + 1]);
                acc[4 * i + 2] = fmaf(w, x[k][i].z, acc[4 * i + 2]);
                acc[4 * i + 3] = fmaf(w, x[k][i].w, acc[4 * i + 3]);
            }
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    if (a.lse && blockIdx.y == 0) a.lse[r * kHq + h] = den == 0.f ? -INFINITY : (M + log2f(den)) * kLn2;
    uint4 w;
    __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (r * kHq + h) * (int64_t)kDv + blockIdx.y * kCols) = w;
}

int box_rows(int page_size) {
    if (!page_size) return kKeys;
    const int b = page_size & -page_size;
    return b < kKeys ? b : kKeys;
}

// clusters that can be resident at once (0: unknown)
int64_t resident_clusters() {
    static int cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cache[dev]) return cache[dev] > 0 ? cache[dev] : 0;
    cudaFuncSetAttribute(dense_mla_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, dense_mla_kernel<false>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    cache[dev] = n > 0 ? n : -1;
    return n > 0 ? n : 0;
}

}  // namespace

bool dense_mla_supported(const DenseArgs& a, int dtype, const Geom& g) {
    return mla_tc_supported(dtype, a.Hq, a.Hkv, a.dk, a.dv, a.k, a.v, a.k_stride, a.kv_rows, a.q, a.out) &&
           a.kv_rows <= INT32_MAX - kKeys && (!g.page_table || box_rows(g.page_size) >= 8);
}

// key splits per query row, as the sparse unit's: the clusters covered once, at least 256 and at most
// kMaxKps keys each
int dense_mla_splits(int64_t n_rows, int64_t max_n_kv) { return mla_splits(n_rows, max_n_kv); }

size_t dense_mla_workspace_bytes(int64_t n_rows, int64_t max_n_kv) { return mla_workspace_bytes(n_rows, max_n_kv); }

cudaError_t launch_dense_mla(const DenseArgs& args, const Geom& g, void* ws, size_t ws_bytes, cudaStream_t st) {
    const int64_t n_rows = (int64_t)g.B * g.T;
    DenseParams p = {args, box_rows(g.page_size), 0};
    DenseArgs& a = p.a;
    int64_t splits = dense_mla_splits(n_rows, g.max_n_kv);
    const int64_t per_split = n_rows * kHq * (kDv + 2) * (int64_t)sizeof(float);
    const int64_t fit = ws ? (int64_t)ws_bytes / per_split : 0;
    if (splits > 1 && splits > fit) splits = fit;
    if (splits < 1) splits = 1;
    int64_t kps = (((int64_t)g.max_n_kv + splits - 1) / splits + kKeys - 1) / kKeys * kKeys;
    if (kps < kKeys) kps = kKeys;
    if (kps > kMaxKps) return cudaErrorNotSupported;      // the workspace holds too few splits
    splits = ((int64_t)g.max_n_kv + kps - 1) / kps;
    if (splits < 1) splits = 1;
    a.splits = (int)splits;
    p.kps = (int)kps;
    a.part_o = splits > 1 ? static_cast<float*>(ws) : nullptr;
    a.part_ml = splits > 1 ? a.part_o + (size_t)n_rows * splits * kHq * kDv : nullptr;
    CUtensorMap map;
    if (!make_head_tmap(&map, a.k, true, kDk, 1, a.k_stride, a.kv_rows, p.box)) return cudaErrorNotSupported;
    const bool mods = a.mods.softcap > 0.f || a.mods.slopes;
    auto kern = mods ? dense_mla_kernel<true> : dense_mla_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    const int64_t n_units = n_rows * splits, resident = resident_clusters();
    const int64_t clusters = resident > 0 && resident < n_units ? resident : n_units;
    if (2 * clusters > INT32_MAX) return cudaErrorNotSupported;
    e = launch_pdl(kern, dim3((unsigned)(2 * clusters)), dim3(kThreads), kSmemBytes, st, p, g, n_units, map);
    if (e != cudaSuccess || splits == 1) return e;
    return launch_pdl(dense_mla_combine_kernel, dim3((unsigned)n_rows, kDv / kCols), dim3(kHq), 0, st, a);
}

}  // namespace lidx
