// Dense attention over a (paged) MLA latent cache on the tensor cores: 128 query
// heads, bf16 rows of 576 columns, value = the first 512 (dense_attn in lidx.h).
//
// The output O [128 heads x 512] f32 fills all of an SM's tensor memory, so a work
// unit (query row, split of its keys) runs on a cluster of two CTAs and walks
// tiles of 64 consecutive positions:
//   rank 0: Q [128 x 576] lies in TMEM; S = Q K^T (two buffers of 64 columns),
//           softmax (thread = head), P = 2^(S*c - m) as bf16, put together in
//           shared memory and sent to rank 1 by a bulk copy per warp;
//   rank 1: O += P V in TMEM (two halves of 256 columns), rescaled when a row's
//           maximum passed its reference by 2^8 (so P stays <= 2^8), and the output.
// K and V rows are the same bytes, loaded by each rank for itself: what one rank
// needs now the other needs a softmax later, and tiles held for both would not fit.
// They come as TMA boxes of at most a page, K in a ring of 24 KB thirds (one is
// loaded again as soon as its products are done), V in one of 32 KB halves, each for
// a product 256 columns wide.
//
// Eight sequences of up to 8192 keys (one token each, 64-row pages): 29 us (972 as plain
// tensor operations): 4 us to the first tile (lengths, page numbers and rows are read
// one after the other), 15 tiles of 64 keys at 1 us, 4 us to write 256 KB of O from each
// SM that holds one, and the launches and the merge.  A tile is bound by rank 0's
// scores: 36 products that take 35 cycles each to issue, and the waits between them,
// which stand where the pipe has work.  64 tokens on 16384 keys each: 297 us = 0.98
// PFLOP/s.
//
// Every head of a query row sees the same keys, so a tile needs one bit per key;
// rows without their bit (a page's unwritten end, a page out of range) are zeroed
// in rank 1's tile before it is multiplied, so that nothing in them reaches the
// output.  Splits are merged by a kernel of their own, which also writes lse.
// P is rounded to bf16 for the product (half a step, averaged over the keys); sums,
// maxima, O and the splits' parts are f32.  Every wait is bounded; a timeout records
// IDX_ERR_TIMEOUT and the cluster winds down.
#include "dense_attn.cuh"
#include "sm100_ptx.cuh"

namespace lidx {
namespace {
using namespace sm100;

constexpr int kHq = 128;
constexpr int kDk = 576;
constexpr int kDv = 512;
constexpr int kKeys = 64;                       // keys per tile
constexpr int kBlockBytes = kKeys * 128;        // 64 columns of a tile
constexpr int kDkBlocks = kDk / 64;             // 9
constexpr int kGroupBytes = 4 * kBlockBytes;    // 256 columns of a tile
constexpr int kKGroup = 3 * kBlockBytes;        // 192 columns of a tile
constexpr int kKGroups = 3;                     // of a tile
constexpr int kKRing = 7;                       // rank 0: groups in flight
constexpr int kVRing = 5;                       // rank 1: groups in flight
constexpr int kPkts = 3;                        // P tiles on their way
constexpr int kPBytes = kHq * kKeys * 2;
// what a packet holds beside P, a piece per softmax warp
struct PktTail {
    float alpha[32];
    float l[32];      // (with the last packet)
    float m[32];
};
constexpr int kPktBytes = (kPBytes + 4 * (int)sizeof(PktTail) + 1023) / 1024 * 1024;
constexpr int kMaxKps = 8192;                   // keys per split, at most (one bit each)
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr int kSCol0 = 320;                     // rank 0: S buffers at 320 and 384 (Q at 0..287)
constexpr float kRescaleLog2 = 8.f;
// rank 0: [K ring][packets]; rank 1: [V ring][packets]
constexpr int kRegion = 223 * 1024;
static_assert(kKRing * kKGroup + kPkts * kPktBytes <= kRegion && kVRing * kGroupBytes + kPkts * kPktBytes <= kRegion, "layouts");
// Q passes through shared memory, a row per head at a pitch whose 16-byte reads do not collide, behind the first
// tile's blocks, so that these are loaded meanwhile
constexpr int kQPitch = kDk * 2 + 16;
constexpr int kQOff = kRegion - kHq * kQPitch;
static_assert(kQOff >= kKGroups * kKGroup, "the first tile's blocks are free of Q");

struct Ctl {
    uint64_t kfull[kKRing], kempty[kKRing];                  // rank 0: group landed / multiplied
    uint64_t sfull[2], sempty[2];                            // rank 0: S written / read
    uint64_t qbulk, qready;                                  // rank 0: Q's rows landed / Q in TMEM
    uint64_t pfree[kPkts];                                   // rank 0: rank 1's packet slot multiplied
    uint64_t vfull[kVRing], vok[kVRing], vempty[kVRing];     // rank 1: group landed / its unseen rows zeroed / multiplied
    uint64_t pfull[kPkts];                                   // rank 1: packet landed
    uint64_t cdone[kPkts];                                   // rank 1: O corrected for the packet
    uint64_t pvdone[kPkts];                                  // rank 1: packet multiplied
    uint64_t bits;                                           // the unit's bits are there
    uint64_t done;                                           // all of the unit's products
    uint32_t tmem_base;
    int abort;
};

// Warp roles.  Both: 1 issues the products, 2..5 (one per TMEM lane quarter) softmax / correction.
// Rank 0: 0, 6, 7 load K, a third of a tile each; 8.. the bits.
// Rank 1: 0 loads V, 6 zeroes unseen rows, 7.. the bits.
__host__ __device__ constexpr int first_bit_warp(uint32_t rank) { return rank == 0 ? 8 : 7; }

constexpr size_t kSmemBytes = 1024 + (size_t)kRegion + kMaxKps / 8 + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory");

struct DenseParams {
    DenseArgs a;
    int box;          // rows per TMA box: 64, or the largest power of two that divides the page
};

struct Unit {
    int64_t r;        // query row
    int b;            // its sequence
    int lo, hi;       // the split's keys that the row sees
    int base;         // position of the first tile (tiles are cuts of the position line)
    int n_tiles;
    int pos;          // the row's position
};

__device__ __forceinline__ void abort_cta(Ctl& c, int* status) {
    *(volatile int*)&c.abort = 1;
    flag(status, IDX_ERR_TIMEOUT);
}

// the whole warp sees the same answer
__device__ __forceinline__ bool warp_aborted(Ctl& c) { return __any_sync(0xffffffffu, *(volatile int*)&c.abort != 0); }

// a unit's barriers, by one warp (a lane per barrier); again: they were another unit's
__device__ __forceinline__ void init(Ctl& c, uint32_t rank, bool again) {
    const int lane = threadIdx.x & 31;
    auto all = [again, lane](uint64_t* bars, int n, int count) {
        if (lane < n) {
            if (again) mbar_inval(bars + lane);
            mbar_init(bars + lane, count);
        }
    };
    if (rank == 0) {
        all(c.kfull, kKRing, 1);
        all(c.kempty, kKRing, 1);
        all(c.sfull, 2, 1);
        all(c.sempty, 2, 4);
        all(&c.qbulk, 1, 1);
        all(&c.qready, 1, 4);
        all(c.pfree, kPkts, 1);
    } else {
        all(c.vfull, kVRing, 1);
        all(c.vok, kVRing, 1);
        all(c.vempty, kVRing, 1);
        all(c.pfull, kPkts, 1);
        all(c.cdone, kPkts, 4);
        all(c.pvdone, kPkts, 1);
    }
    all(&c.bits, 1, kThreads / 32 - first_bit_warp(rank));
    all(&c.done, 1, 1);
    c.abort = 0;
    fence_mbar_init();
}

// cache row of piece pc of tile t (a box of the tile that one page holds); past the cache, where TMA reads
// zeros, for a piece without a key to see.  (Rows that a wild page number leads to are not seen either.)
__device__ __forceinline__ int piece_row(const DenseParams& p, const Unit& u, const Geom& g, int t, int pc) {
    const int j = u.base + t * kKeys + pc * p.box;
    int64_t row = p.a.kv_rows;
    if (t < u.n_tiles && j + p.box > u.lo && j < u.hi) {
        row = key_row(g, u.b, j);
        if (row > p.a.kv_rows) row = p.a.kv_rows;
        if (row < -kKeys) row = -kKeys;
    }
    return (int)row;
}

// one bit per key of the unit's tiles
__device__ __forceinline__ void stage_bits(Ctl& c, uint32_t* vmask, uint32_t rank, const Unit& u, const Geom& g, int64_t kv_rows) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = first_bit_warp(rank);
    for (int w = warp - first; w < u.n_tiles * (kKeys / 32); w += kThreads / 32 - first) {
        const int j = u.base + w * 32 + lane;
        bool seen = j >= u.lo && j < u.hi;
        if (seen) {
            const int64_t row = key_row(g, u.b, j);
            if (row < 0 || row >= kv_rows) {
                seen = false;
                if (rank == 0) flag(g.status, IDX_ERR_DEVICE_BOUNDS);
            }
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, seen);
        if (lane == 0) vmask[w] = bits;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.bits);
}

// rank 0, warps 2..5 (thread = head): Q of the unit's row into TMEM columns 0..287, the score product's A operand
__device__ __forceinline__ void load_q(Ctl& c, uint8_t* smem, uint32_t tmem, const void* q, const Unit& u, int* status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = (warp & 3) * 32 + lane;
    uint8_t* row = smem + kQOff + h * kQPitch;
    if (warp == 2 && lane == 0) mbar_arrive_expect_tx(&c.qbulk, kHq * kDk * 2);
    bulk_load(row, static_cast<const __nv_bfloat16*>(q) + (u.r * kHq + h) * (int64_t)kDk, kDk * 2, &c.qbulk);
    if (!warp_wait(&c.qbulk, 0)) abort_cta(c, status);
    const uint4* src = reinterpret_cast<const uint4*>(row);
#pragma unroll
    for (int cb = 0; cb < kDkBlocks; ++cb) {
        uint32_t regs[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 x = src[cb * 8 + i];
            regs[4 * i] = x.x;
            regs[4 * i + 1] = x.y;
            regs[4 * i + 2] = x.z;
            regs[4 * i + 3] = x.w;
        }
        tmem_st_32x32b_x32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + cb * 32, regs);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.qready);
}

// rank 0, loader li: its group of every tile
__device__ __forceinline__ void load_k(Ctl& c, uint8_t* ring, const CUtensorMap* map, const DenseParams& p, const Unit& u,
                                       const Geom& g, int li) {
    const int lane = threadIdx.x & 31, pieces = kKeys / p.box;
    const int pc = lane % pieces, cb = lane / pieces;      // (at most 8 pieces: three blocks' are at most 24)
    bool ok = true;
    int sent = 0;
    fence_proxy_async_smem();    // what was read or written here before is done with
    int row = piece_row(p, u, g, 0, pc);
    for (int t = 0; ok && t < u.n_tiles; ++t) {
        const int next = piece_row(p, u, g, t + 1, pc);     // (its latency under this tile's waits)
        if (t == 1) {
            ok = warp_wait(&c.qready, 0);      // Q passed through the blocks that follow
            fence_proxy_async_smem();
        }
        const int i = t * kKGroups + li, slot = i % kKRing;
        ok = ok && !warp_aborted(c) && warp_wait(&c.kempty[slot], (uint32_t)((i / kKRing) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&c.kfull[slot], kKGroup);
        __syncwarp();
        if (cb < 3)
            tma_load_3d(ring + slot * kKGroup + cb * kBlockBytes + pc * p.box * 128, map, &c.kfull[slot], (li * 3 + cb) * 64, 0,
                        row);
        sent = t + 1;
        row = next;
    }
    if (!ok) {
        abort_cta(c, g.status);     // no load may still be in flight when the CTA ends
        for (int t = max(0, sent - 1 - kKRing / kKGroups); t < sent; ++t) {
            const int i = t * kKGroups + li;
            if (i + kKRing > (sent - 1) * kKGroups + li) warp_wait(&c.kfull[i % kKRing], (uint32_t)((i / kKRing) & 1));
        }
    }
}

// rank 1, one warp: the value groups of every tile
__device__ __forceinline__ void load_v(Ctl& c, uint8_t* ring, const CUtensorMap* map, const DenseParams& p, const Unit& u,
                                       const Geom& g) {
    const int lane = threadIdx.x & 31, pieces = kKeys / p.box;
    const int pc = lane % pieces, cb = lane / pieces;      // (at most 8 pieces: four blocks' are at most 32)
    bool ok = true;
    int sent = 0;
    fence_proxy_async_smem();    // what was read or written here before is done with
    int row = piece_row(p, u, g, 0, pc);
    for (int t = 0; ok && t < u.n_tiles; ++t) {
        const int next = piece_row(p, u, g, t + 1, pc);
        for (int nh = 0; nh < 2; ++nh) {
            const int i = 2 * t + nh, slot = i % kVRing;
            ok = !warp_aborted(c) && warp_wait(&c.vempty[slot], (uint32_t)((i / kVRing) & 1) ^ 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&c.vfull[slot], kGroupBytes);
            __syncwarp();
            if (cb < 4)
                tma_load_3d(ring + slot * kGroupBytes + cb * kBlockBytes + pc * p.box * 128, map, &c.vfull[slot],
                            (nh * 4 + cb) * 64, 0, row);
            sent = i + 1;
        }
        row = next;
    }
    if (!ok) {
        abort_cta(c, g.status);
        for (int i = max(0, sent - kVRing); i < sent; ++i) warp_wait(&c.vfull[i % kVRing], (uint32_t)((i / kVRing) & 1));
    }
}

// rank 1, one warp: zero the value rows that are not seen
__device__ __forceinline__ void zero_unseen(Ctl& c, uint8_t* ring, const Unit& u, const uint32_t* vmask, const Geom& g) {
    const int lane = threadIdx.x & 31;
    bool ok = warp_wait(&c.bits, 0);
    for (int i = 0; ok && i < 2 * u.n_tiles; ++i) {
        const int slot = i % kVRing, t = i >> 1;
        ok = !warp_aborted(c) && warp_wait(&c.vfull[slot], (uint32_t)((i / kVRing) & 1));
        if (!ok) break;
        const uint64_t seen = (uint64_t)vmask[2 * t] | (uint64_t)vmask[2 * t + 1] << 32;
        if (seen != ~0ull) {
            for (int e = lane; e < kKeys * 4 * 8; e += 32) {
                const int row = (e >> 3) & (kKeys - 1), cb = e / (kKeys * 8);
                if (!((seen >> row) & 1ull))
                    *reinterpret_cast<uint4*>(ring + slot * kGroupBytes + cb * kBlockBytes + row * 128 + (e & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
        }
        if (lane == 0) mbar_arrive(&c.vok[slot]);
    }
    if (!ok) abort_cta(c, g.status);
}

// The issuers walk as a warp and a lane issues: operands that all lanes share stay in uniform registers (a lane on
// its own takes about 100 cycles for each product, which takes 33).
__device__ __forceinline__ void issue_qk(Ctl& c, const uint8_t* ring, uint32_t tmem, const Unit& u, const Geom& g) {
    const uint32_t idesc = idesc_f16_f32_major(kHq, kKeys, 1, 0, 0);
    const uint64_t kd = desc_sw128_kmajor(0, 1024);
    const uint32_t k_hi = desc_hi(kd), tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t kb = (uint32_t)kd + desc_addr(ring);
    bool ok = u.n_tiles == 0 || warp_wait(&c.qready, 0);
    int slot = 0;
    uint32_t phase = 0;
    ok = ok && (u.n_tiles == 0 || (warp_wait(&c.sempty[0], 1u) && warp_wait(&c.kfull[0], 0u)));
    for (int t = 0; ok && t < u.n_tiles; ++t) {
        const int sb = t & 1;
        const uint32_t d = __shfl_sync(0xffffffffu, tm + kSCol0 + sb * kKeys, 0);
#pragma unroll
        for (int kg = 0; kg < kKGroups; ++kg) {
            const uint32_t ka = __shfl_sync(0xffffffffu, kb + (slot * kKGroup >> 4), 0);
            const uint32_t now = (uint32_t)slot;
            if (++slot == kKRing) {
                slot = 0;
                phase ^= 1;
            }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 6; ++ks)
                    mma_f16_ts_lo(d, tm + (kg * 12 + ks) * 8, ka + (((ks >> 2) * kBlockBytes + (ks & 3) * 32) >> 4), k_hi, idesc,
                                  kg + ks > 0 ? 1u : 0u);
            }
            __syncwarp();
            // the next third's wait, while the pipe has work
            if (kg < kKGroups - 1)
                ok = warp_wait(&c.kfull[slot], phase);
            else if (t + 1 < u.n_tiles)
                ok = warp_wait(&c.kfull[slot], phase) && warp_wait(&c.sempty[sb ^ 1], (uint32_t)(((t + 1) >> 1) & 1) ^ 1);
            if (!ok) break;
            if (elect_one()) {
#pragma unroll
                for (int ks = 6; ks < 12; ++ks)
                    mma_f16_ts_lo(d, tm + (kg * 12 + ks) * 8, ka + (((ks >> 2) * kBlockBytes + (ks & 3) * 32) >> 4), k_hi, idesc, 1u);
                mma_commit(&c.kempty[now]);
                if (kg == kKGroups - 1) mma_commit(&c.sfull[sb]);
            }
            __syncwarp();
        }
    }
    if (!ok) abort_cta(c, g.status);
    if (elect_one()) mma_commit(&c.done);
    __syncwarp();
    warp_wait(&c.done, 0);
}

__device__ __forceinline__ void issue_pv(Ctl& c, const uint8_t* ring, const uint8_t* pkts, uint32_t tmem, const Unit& u,
                                         const Geom& g) {
    const uint32_t idesc = idesc_f16_f32_major(kHq, 256, 1, 0, 1);
    const uint64_t pd = desc_sw128_kmajor(0, 1024), vd = desc_sw128_mnmajor(0, kBlockBytes, 1024);
    const uint32_t p_hi = desc_hi(pd), v_hi = desc_hi(vd), tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t pb = (uint32_t)pd + desc_addr(pkts), vb = (uint32_t)vd + desc_addr(ring);
    bool ok = true;
    for (int t = 0; ok && t < u.n_tiles; ++t) {
        const int j = t % kPkts;
        ok = warp_wait(&c.cdone[j], (uint32_t)((t / kPkts) & 1));
        const uint32_t pa = __shfl_sync(0xffffffffu, pb + (j * kPktBytes >> 4), 0);
        const uint32_t acc = __shfl_sync(0xffffffffu, t > 0 ? 1u : 0u, 0);
#pragma unroll
        for (int nh = 0; nh < 2; ++nh) {
            const int i = 2 * t + nh, slot = i % kVRing;
            ok = ok && warp_wait(&c.vok[slot], (uint32_t)((i / kVRing) & 1));
            fence_proxy_async_smem();
            tc_fence_after();
            const uint32_t va = __shfl_sync(0xffffffffu, vb + (slot * kGroupBytes >> 4), 0);
            if (ok && elect_one()) {
#pragma unroll
                for (int ks = 0; ks < kKeys / 16; ++ks)
                    mma_f16_ss_lo(tm + nh * 256, pa + (ks * 32 >> 4), p_hi, va + (ks * 2 * 1024 >> 4), v_hi, idesc,
                                  ks > 0 ? 1u : acc);
                mma_commit(&c.vempty[slot]);
                if (nh == 1) {
                    mma_commit(&c.pvdone[j]);
                    mma_commit_multicast(&c.pfree[j], (uint16_t)0x1);
                }
            }
            __syncwarp();
        }
    }
    if (!ok) abort_cta(c, g.status);
    if (elect_one()) mma_commit(&c.done);
    __syncwarp();
    warp_wait(&c.done, 0);
}

// rank 0, warps 2..5 (thread = head)
template <bool kMods>
__device__ __forceinline__ void softmax(Ctl& c, uint8_t* smem, uint32_t tmem, const DenseParams& p, const Unit& u,
                                        const uint32_t* vmask, const Geom& g) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3;
    const int h = quad * 32 + lane;
    const uint32_t s_col = tmem + ((uint32_t)(quad * 32) << 16) + kSCol0;
    uint8_t* own = smem + kKRing * kKGroup;
    const uint32_t pkts = mapa(smem + kVRing * kGroupBytes, 1);
    const float sl2 = kMods ? 1.f : p.a.scale * kLog2e;
    Score sc;
    if (kMods) sc = make_score(p.a, p.a.mods.slopes ? p.a.mods.slopes[h] : 0.f);
    float m_used = 0.f, lsum = 0.f;
    bool has_m = false;
    bool ok = warp_wait(&c.bits, 0);
    for (int t = 0; ok && t < u.n_tiles; ++t) {
        const int sb = t & 1, j = t % kPkts;
        const uint32_t ma = vmask[2 * t], mb = vmask[2 * t + 1];
        ok = !warp_aborted(c) && warp_wait(&c.sfull[sb], (uint32_t)((t >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
        float s0[32], s1[32];
        tmem_ld_32x32b_x32(s_col + sb * kKeys, s0);
        tmem_ld_32x32b_x32(s_col + sb * kKeys + 32, s1);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.sempty[sb]);
        if constexpr (kMods) {      // scores in log2 units
            const int j0 = u.base + t * kKeys;
            const float d = (float)(u.pos - j0);
            const bool past = j0 + kKeys <= u.pos + 1;      // (every head of the row alike)
            modify(s0, sc, d, past);
            modify(s1, sc, d - 32.f, past);
        }
        // the tile's largest scaled score: for a full tile and a positive scale, the scaled largest score (the same
        // value: rounding a product by a positive factor is monotone)
        const bool full = (ma & mb) == 0xffffffffu;
        float mt = -3.0e38f;
        if (full && sl2 > 0.f) {
            float a0 = fmaxf(s0[0], s0[1]), a1 = fmaxf(s0[2], s0[3]);
            float a2 = fmaxf(s1[0], s1[1]), a3 = fmaxf(s1[2], s1[3]);
#pragma unroll
            for (int i = 4; i < 32; i += 4) {
                a0 = fmaxf(a0, fmaxf(s0[i], s0[i + 1]));
                a1 = fmaxf(a1, fmaxf(s0[i + 2], s0[i + 3]));
                a2 = fmaxf(a2, fmaxf(s1[i], s1[i + 1]));
                a3 = fmaxf(a3, fmaxf(s1[i + 2], s1[i + 3]));
            }
            mt = fmaxf(mt, fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * sl2);     // (finite where every score is -inf)
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if ((ma >> i) & 1u) mt = fmaxf(mt, s0[i] * sl2);
                if ((mb >> i) & 1u) mt = fmaxf(mt, s1[i] * sl2);
            }
        }
        float alpha = 1.f;
        if ((ma | mb) != 0u) {
            if (!has_m) {
                m_used = mt;
                has_m = true;
            } else if (mt > m_used + kRescaleLog2) {
                alpha = ex2_approx(m_used - mt);
                lsum *= alpha;
                m_used = mt;
            }
        }
        // p = 2^(s * scale_log2 - m) with one rounding of the exponent's argument (FMA)
        uint32_t pk[32];
        float psum = 0.f;
        const float nm = -m_used;
        auto weights = [&](auto all) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float e0 = ex2_approx(fmaf(s0[2 * i], sl2, nm)), e1 = ex2_approx(fmaf(s0[2 * i + 1], sl2, nm));
                float e2 = ex2_approx(fmaf(s1[2 * i], sl2, nm)), e3 = ex2_approx(fmaf(s1[2 * i + 1], sl2, nm));
                if (!decltype(all)::value) {
                    e0 = ((ma >> (2 * i)) & 1u) ? e0 : 0.f;
                    e1 = ((ma >> (2 * i + 1)) & 1u) ? e1 : 0.f;
                    e2 = ((mb >> (2 * i)) & 1u) ? e2 : 0.f;
                    e3 = ((mb >> (2 * i + 1)) & 1u) ? e3 : 0.f;
                }
                psum += (e0 + e1) + (e2 + e3);
                const __nv_bfloat162 x = __floats2bfloat162_rn(e0, e1), y = __floats2bfloat162_rn(e2, e3);
                pk[i] = *reinterpret_cast<const uint32_t*>(&x);
                pk[16 + i] = *reinterpret_cast<const uint32_t*>(&y);
            }
        };
        if (full)
            weights(std::true_type{});
        else
            weights(std::false_type{});
        lsum += psum;

        // slot j, here and in rank 1, is free once rank 1's products of tile t - kPkts are done
        ok = warp_wait(&c.pfree[j], (uint32_t)((t / kPkts) & 1) ^ 1);
        if (!ok) break;
        const uint32_t rbar = mapa(&c.pfull[j], 1);
        const bool totals = t == u.n_tiles - 1;      // the sum and the reference go with the last packet
        // the warp's 32 rows are 4 KB of the tile: put together here, one copy sends them, a second their factors.  (Each
        // store into rank 1 that completes a transaction of a barrier takes its place there for about three cycles: a
        // thread's 16-byte pieces, 1152 a tile, took 3500.)
        uint8_t* rows = own + j * kPktBytes + quad * (kPBytes / 4);
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
            *reinterpret_cast<uint4*>(rows + lane * 128 + ((ch ^ (lane & 7)) << 4)) =
                make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
        float* mine = reinterpret_cast<float*>(own + j * kPktBytes + kPBytes + quad * (int)sizeof(PktTail));
        mine[lane] = alpha;
        if (totals) {
            mine[32 + lane] = lsum;
            mine[64 + lane] = m_used;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            bulk_copy_to_cta(pkts + j * kPktBytes + quad * (kPBytes / 4), rows, kPBytes / 4, rbar);
            bulk_copy_to_cta(pkts + j * kPktBytes + kPBytes + quad * (uint32_t)sizeof(PktTail), mine,
                             (uint32_t)sizeof(PktTail) / (totals ? 1 : 3), rbar);
        }
    }
    if (!ok) abort_cta(c, g.status);
    // rank 1's last arrivals on pfree land before this CTA may leave (and its packets have left its memory)
    for (int t = max(0, u.n_tiles - kPkts); t < u.n_tiles; ++t)
        if (!warp_aborted(c)) warp_wait(&c.pfree[t % kPkts], (uint32_t)((t / kPkts) & 1));
    if (warp_aborted(c))
        for (int i = 0; i < 50; ++i) __nanosleep(1000);      // ample for 4 KB to the neighbour
}

// rank 1, warps 2..5 (thread = head): O follows its rows' references
__device__ __forceinline__ void correct(Ctl& c, const uint8_t* pkts, uint32_t tmem, const Unit& u, const Geom& g) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    bool ok = true;
    for (int t = 0; ok && t < u.n_tiles; ++t) {
        const int j = t % kPkts;
        // (announced here: an arrival from rank 0 would have to wait there for all that the thread sent before, 2000 cycles)
        if (warp == 2 && lane == 0) mbar_arrive_expect_tx(&c.pfull[j], kPBytes + kHq * 4 * (t == u.n_tiles - 1 ? 3 : 1));
        ok = !warp_aborted(c) && warp_wait_cluster(&c.pfull[j], (uint32_t)((t / kPkts) & 1));
        if (!ok) break;
        const float a = reinterpret_cast<const PktTail*>(pkts + j * kPktBytes + kPBytes)[quad].alpha[lane];
        if (t > 0 && __any_sync(0xffffffffu, a != 1.f)) {
            ok = warp_wait(&c.pvdone[(t - 1) % kPkts], (uint32_t)(((t - 1) / kPkts) & 1));
            if (!ok) break;
            tc_fence_after();
            for (int cb = 0; cb < kDv / 32; ++cb) {
                float v[32];
                tmem_ld_32x32b_x32(tmem + lane_off + cb * 32, v);
                tmem_ld_wait();
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i] * a);
                tmem_st_32x32b_x32(tmem + lane_off + cb * 32, w);
            }
            tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.cdone[j]);
    }
    if (!ok) abort_cta(c, g.status);
}

// rank 1, every warp: three to a TMEM lane quarter (thread = head), each every third 32 columns
__device__ __forceinline__ void output(Ctl& c, uint8_t* smem, uint32_t tmem, const DenseArgs& a, const Unit& u, int64_t unit,
                                       const Geom& g) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, part = warp >> 2;
    const int h = quad * 32 + lane;
    const uint32_t o_col = tmem + ((uint32_t)(quad * 32) << 16);
    float lsum = 0.f, mrow = 0.f;
    bool have = u.n_tiles > 0 && !warp_aborted(c);
    if (have && !warp_wait(&c.done, 0u)) {
        abort_cta(c, g.status);
        have = false;
    }
    if (have) {
        tc_fence_after();
        const PktTail& tail = reinterpret_cast<const PktTail*>(smem + kVRing * kGroupBytes + (u.n_tiles - 1) % kPkts * kPktBytes +
                                                               kPBytes)[quad];
        lsum = tail.l[lane];
        mrow = tail.m[lane];
    }
    auto columns = [&](int cb, float (&v)[32]) {
        if (have) {
            tmem_ld_32x32b_x32(o_col + cb * 32, v);
            tmem_ld_wait();
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
    };
    if (a.part_o) {
        // [unit][column / 4][head][4]: for each four columns the warp's 32 heads are 512 contiguous bytes
        float4* po = reinterpret_cast<float4*>(a.part_o + unit * (int64_t)kDv * kHq) + h;
        for (int cb = part; cb < kDv / 32; cb += kThreads / 128) {
            float v[32];
            columns(cb, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) po[(int64_t)(cb * 8 + i) * kHq] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        if (part == 0) reinterpret_cast<float2*>(a.part_ml)[unit * kHq + h] = make_float2(mrow, lsum);
        return;
    }
    // (a NaN sum passes the test: the row is NaN then)
    const float inv = lsum != 0.f ? 1.f / lsum : 0.f;
    if (a.lse && part == 0) a.lse[u.r * kHq + h] = lsum == 0.f ? -INFINITY : (mrow + log2f(lsum)) * kLn2;
    // the warp's 32 heads x 32 columns pass through shared memory (the idle value ring; rows of 80 bytes), so that a
    // store instruction writes eight heads' 64-byte segments whole
    uint8_t* tw = smem + warp * (32 * 80);
    __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(a.out) + (u.r * kHq + quad * 32) * (int64_t)kDv;
    for (int cb = part; cb < kDv / 32; cb += kThreads / 128) {
        float v[32];
        columns(cb, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 w;
            __nv_bfloat162* b2 = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
            for (int e = 0; e < 4; ++e) b2[e] = __floats2bfloat162_rn(v[8 * i + 2 * e] * inv, v[8 * i + 2 * e + 1] * inv);
            *reinterpret_cast<uint4*>(tw + lane * 80 + i * 16) = w;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rr = 8 * i + (lane >> 2), ch = lane & 3;
            *reinterpret_cast<uint4*>(ob + (int64_t)rr * kDv + cb * 32 + ch * 8) =
                *reinterpret_cast<const uint4*>(tw + rr * 80 + ch * 16);
        }
        __syncwarp();
    }
}

template <bool kMods>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_mla_kernel(DenseParams p, Geom g, int n_units, const __grid_constant__ CUtensorMap map) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t* vmask = reinterpret_cast<uint32_t*>(smem + kRegion);
    Ctl& c = *reinterpret_cast<Ctl*>(vmask + kMaxKps / 32);
    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x >> 5;
    const int n_clusters = gridDim.x >> 1;
    const DenseArgs& a = p.a;
    if (a.part_o) pdl_trigger();     // (the merge follows; results are not handed on early, see lidx_internal.cuh)
    if (warp == 0) init(c, rank, false);
    if (threadIdx.x == 0) tma_prefetch_desc(&map);
    if (warp == 1) {
        tmem_alloc(&c.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem_base;
    pdl_wait();
    for (int64_t next = blockIdx.x >> 1; next < n_units; next += n_clusters) {
        const int unit = (int)next;
        cluster_arrive();      // (this CTA's barriers are ready)
        Unit u;
        const int row = unit / a.splits;
        u.r = row;
        u.b = row / g.T;
        const Interval iv = row_interval(g, a.mods, u.r, u.b, seq_n_kv(g, u.b));
        // the split's share of the tiles (cuts of the position line) that the row sees part of
        const int first = iv.lo / kKeys, seen = iv.hi > iv.lo ? (iv.hi + kKeys - 1) / kKeys - first : 0;
        const int share = (seen + a.splits - 1) / a.splits, at = min((unit - row * a.splits) * share, seen);
        u.base = (first + at) * kKeys;
        u.n_tiles = max(0, min(share, seen - at));
        u.lo = max(iv.lo, u.base);
        u.hi = min(iv.hi, u.base + u.n_tiles * kKeys);
        u.pos = iv.pos;
        // (what loads and what looks at page numbers does not wait for the other CTA)
        if (rank == 0) {
            if (warp == 0 || warp == 6 || warp == 7) {
                load_k(c, smem, &map, p, u, g, warp == 0 ? 0 : warp - 5);
                cluster_wait();
            } else if (warp >= first_bit_warp(0)) {
                stage_bits(c, vmask, rank, u, g, a.kv_rows);
                cluster_wait();
            } else if (warp == 1) {
                cluster_wait();
                issue_qk(c, smem, tmem, u, g);
            } else {
                if (u.n_tiles > 0) load_q(c, smem, tmem, a.q, u, g.status);
                cluster_wait();
                softmax<kMods>(c, smem, tmem, p, u, vmask, g);
            }
        } else {
            if (warp == 0) load_v(c, smem, &map, p, u, g);
            else if (warp >= first_bit_warp(1)) stage_bits(c, vmask, rank, u, g, a.kv_rows);
            cluster_wait();
            if (warp == 1) issue_pv(c, smem, smem + kVRing * kGroupBytes, tmem, u, g);
            else if (warp >= 2 && warp <= 5) correct(c, smem + kVRing * kGroupBytes, tmem, u, g);
            else if (warp == 6) zero_unseen(c, smem, u, vmask, g);
            output(c, smem, tmem, a, u, unit, g);
        }
        tc_fence_before();
        __syncthreads();
        // (nothing of the other CTA's is on its way to this one's barriers: what it sent has been waited for)
        if (warp == 0 && next + n_clusters < n_units) init(c, rank, true);
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
    // kBatch splits at a time, all of their loads in flight together (a call rarely has more: one pass)
    constexpr int kBatch = 16;
    float M = -INFINITY, acc[kCols], den = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
    for (int s0 = 0; s0 < a.splits; s0 += kBatch) {
        float2 ml[kBatch];
        float4 x[kBatch][kCols / 4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            ml[k] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i) x[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s0 + k >= a.splits) continue;
            const int64_t u = r * a.splits + s0 + k;
            ml[k] = reinterpret_cast<const float2*>(a.part_ml)[u * kHq + h];
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i)
                x[k][i] = reinterpret_cast<const float4*>(a.part_o + u * (int64_t)kDv * kHq)[(int64_t)(blockIdx.y * (kCols / 4) + i) * kHq + h];
        }
        float m_new = M;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (ml[k].y != 0.f) m_new = fmaxf(m_new, ml[k].x);
        const float old = M == m_new ? 1.f : exp2f(M - m_new);
        M = m_new;
        den *= old;
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] *= old;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const bool in = ml[k].y != 0.f;      // (a split without keys wrote zeros)
            const float w = in ? exp2f(ml[k].x - M) : 0.f;
            den += in ? w * ml[k].y : 0.f;
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i) {
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
           a.kv_rows <= INT32_MAX - kKeys && (!g.page_table || box_rows(g.page_size, kKeys) >= 8);
}

// key splits per query row: the fewest rounds of the clusters x tiles of a unit, which has about 10 tiles' time of
// its own (Q, the first loads, the output); at least 256 and at most kMaxKps keys each
int dense_mla_splits(int64_t n_rows, int64_t max_n_kv) {
    const int64_t min_s = max_n_kv > kMaxKps ? (max_n_kv + kMaxKps - 1) / kMaxKps : 1;
    if (n_rows <= 0) return (int)min_s;
    const int sms = sm_count();
    const int64_t clusters = sms < 2 ? 76 : sms / 2;
    const int64_t tiles = (max_n_kv + kKeys - 1) / kKeys;
    auto cost = [&](int64_t s) { return (n_rows * s + clusters - 1) / clusters * ((tiles + s - 1) / s + 10); };
    int64_t best = min_s;
    for (int64_t s = min_s + 1; s <= clusters && s * 256 <= max_n_kv + 255; ++s)
        if (cost(s) < cost(best)) best = s;
    return (int)best;
}

size_t dense_mla_workspace_bytes(int64_t n_rows, int64_t max_n_kv) {
    const int s = dense_mla_splits(n_rows, max_n_kv);
    return s <= 1 ? 0 : (size_t)n_rows * s * kHq * (kDv + 2) * sizeof(float);
}

cudaError_t launch_dense_mla(const DenseArgs& args, const Geom& g, void* ws, size_t ws_bytes, cudaStream_t st) {
    const int64_t n_rows = (int64_t)g.B * g.T;
    DenseParams p = {args, box_rows(g.page_size, kKeys)};
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
    a.part_o = splits > 1 ? static_cast<float*>(ws) : nullptr;
    a.part_ml = splits > 1 ? a.part_o + (size_t)n_rows * splits * kHq * kDv : nullptr;
    CUtensorMap map;
    if (!make_head_tmap(&map, a.k, true, kDk, 1, a.k_stride, a.kv_rows, p.box)) return cudaErrorNotSupported;
    const bool mods = a.mods.softcap > 0.f || a.mods.slopes;
    auto kern = mods ? dense_mla_kernel<true> : dense_mla_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    const int64_t n_units = n_rows * splits, resident = resident_clusters();
    if (n_units > INT32_MAX) return cudaErrorNotSupported;
    const int64_t clusters = resident > 0 && resident < n_units ? resident : n_units;
    if (2 * clusters > INT32_MAX) return cudaErrorNotSupported;
    e = launch_pdl(kern, dim3((unsigned)(2 * clusters)), dim3(kThreads), kSmemBytes, st, p, g, (int)n_units, map);
    if (e != cudaSuccess || splits == 1) return e;
    return launch_pdl(dense_mla_combine_kernel, dim3((unsigned)n_rows, kDv / kCols), dim3(kHq), 0, st, a);
}

}  // namespace lidx
