// Dense attention over (paged) caches on the CUDA cores (dense_attn in lidx.h):
// every type, head layout, width and alignment, and all of f32.
//
// The T query rows and the G = Hq / Hkv heads that share kv head g are packed
// into rows m = t*G + h, so that a tile of R packed rows reads each K and V row
// once for all of them.  A CTA of 128 threads owns R rows (64 for wide chunks,
// 16 for few rows or values wider than 128) and one split of its keys, and
// walks it in tiles of 32 keys held in shared memory as f32:
//   scores: thread = (row group, key group), a register block of 4 rows x
//           (R/16) keys fed by 16-byte reads; masked by the rows' intervals;
//   softmax: running maximum and sum per row (natural logarithm), f32;
//   values: thread = (row group, 4-column groups), a register block of the
//           output rescaled by the rows' factors each tile.
// A warp has the same R/4 rows in all three, so that only the tiles' arrival is a barrier of the CTA.
// Sums, products, maxima and weights are f32 throughout; products run as packed pairs of FMAs.
// Measured in f32: 512 tokens on 4096 cached keys, two sequences of 32 heads of 128 on 4, 2.39 ms = 27.0 TFLOP/s.  The
// FMA pipe is active on 41 % of the cycles and a scheduler issues on 35 %: its two warps (two CTAs of four to an SM, all
// that 252 registers and 110 KB leave room for) wait for results and for shared memory.  One token on 16384 keys, eight
// sequences of 32 heads on 8: 0.59 ms = 1.8 TB/s, bound by the latency of a tile's loads and its softmax.
// Loading a tile ahead of the arithmetic (f32, aligned): heads of 64, 256 tokens on 2048 keys 260 -> 194 us.
// A key that only some rows of a tile see is skipped, not multiplied by zero,
// for the others, so that NaN or infinity in it cannot reach them.
#include <float.h>

#include "dense_attn.cuh"

namespace lidx {
namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 32;

__host__ __device__ constexpr int round_up(int x, int m) { return (x + m - 1) / m * m; }

template <int R, int DV>
struct Shape {
    static constexpr int kKeyGroups = R == 64 ? 8 : 32;      // threads along the keys (scores)
    static constexpr int kRowStep = 32 / kKeyGroups;         // a thread's four rows are this far apart
    static constexpr int kKeysPer = kKeys / kKeyGroups;
    static constexpr int kColGroups = R == 64 ? 16 : 32;     // threads along the columns (values)
    static constexpr int kRowsPer = R / (kThreads / kColGroups);
    static constexpr int kCol4 = DV / (4 * kColGroups);      // 4-column groups per thread
    static_assert(kThreads / kKeyGroups * 4 == R && kRowsPer % 4 == 0 && kCol4 >= 1, "thread layout");
};

// bufs: K and V tiles in flight (2: the next one is loaded under this one's arithmetic).  The rows' statistics come
// first; the merge of key splits lays R rows of dv over Q, K, V and the scores, which narrow keys beside wide values are
// shorter than.
size_t smem_bytes(int R, int DV, int dk, int dv, bool latent, int bufs) {
    const int kp = round_up(dk, 4) + 4;
    const int vp = DV + 4;
    const int walk = R * kp + bufs * kKeys * (kp + (latent ? 0 : vp)) + kKeys * (R + 4);
    return sizeof(int64_t) * kKeys * 2 + (sizeof(float) * 2 + sizeof(int) * 3) * R +
           sizeof(float) * (walk > R * dv ? walk : R * dv);
}

// kAhead (f32, 16-byte aligned rows and widths): K and V go straight to shared memory by asynchronous copies, a tile
// ahead.  Otherwise each tile is loaded, widened and stored before its arithmetic.
// Narrow values: registers for three CTAs to an SM (256 tokens on 2048 keys, heads of 64: 193 -> 187 us); for 128 columns
// neither shared memory nor registers leave room for a third.  There, and for the widest values, the compiler is told of
// two, which it makes use of: 252 registers for 186 (512 tokens on 4096 keys: 2.48 -> 2.39 ms), 223 for 167 (256 tokens on
// 2048 keys, heads of 256: 1.88 -> 1.80 ms).
template <typename T, int R, int DV, bool kAhead>
__global__ void __launch_bounds__(kThreads, DV == 64 ? 3 : DV == 512 || (R == 64 && kAhead) ? 2 : 0)
    dense_generic_kernel(DenseArgs a, Geom g, int tiles, bool vec) {
    using S = Shape<R, DV>;
    extern __shared__ __align__(16) unsigned char sm_raw[];
    const int kp = round_up(a.dk, 4) + 4;       // K and Q pitch: rows 4 banks apart
    const bool latent = a.v == nullptr;
    const int vp = latent ? kp : DV + 4;
    constexpr int kBufs = kAhead ? 2 : 1;
    int64_t* rows_all = reinterpret_cast<int64_t*>(sm_raw);     // [2][kKeys] cache rows, negative: none
    float* alpha_s = reinterpret_cast<float*>(rows_all + 2 * kKeys);   // [R]
    float* slope_s = alpha_s + R;                               // [R]
    int* lo_s = reinterpret_cast<int*>(slope_s + R);
    int* hi_s = lo_s + R;
    int* pos_s = hi_s + R;
    float* qs = reinterpret_cast<float*>(pos_s + R);            // [R][kp]
    float* ks_all = qs + R * kp;                                // [kBufs][kKeys][kp]
    float* vs_all = ks_all + kBufs * kKeys * kp;                // [kBufs][kKeys][vp], unless latent
    float* ss = latent ? vs_all : vs_all + kBufs * kKeys * vp;  // [kKeys][R + 4] scores, then weights

    const int tid = threadIdx.x;
    const int G = a.Hq / a.Hkv;
    int64_t u = blockIdx.x;
    const int split = (int)(u % a.splits);
    u /= a.splits;
    const int tile = (int)(u % tiles);
    u /= tiles;
    const int gkv = (int)(u % a.Hkv);
    const int b = (int)(u / a.Hkv);
    const int64_t m0 = (int64_t)tile * R;        // first packed row
    const int64_t m_end = (int64_t)g.T * G;
    if (a.part_o) pdl_trigger();     // (the merge follows; results are not handed on early, see lidx_internal.cuh)
    pdl_wait();
    const int n_kv = seq_n_kv(g, b);

    // the rows' intervals, and the CTA's: the keys that some row sees
    if (tid < R) {
        const int64_t m = m0 + tid;
        Interval iv = {0, 0, 0};
        float slope = 0.f;
        if (m < m_end) {
            const int t = (int)(m / G), h = gkv * G + (int)(m % G);
            iv = row_interval(g, a.mods, (int64_t)b * g.T + t, b, n_kv);
            if (a.mods.slopes) slope = a.mods.slopes[h];
        }
        lo_s[tid] = iv.lo;
        hi_s[tid] = iv.hi;
        pos_s[tid] = iv.pos;
        slope_s[tid] = slope;
    }
    for (int i = tid; i < R * kp; i += kThreads) {
        const int rr = i / kp, c = i % kp;
        const int64_t m = m0 + rr;
        float x = 0.f;
        if (m < m_end && c < a.dk)
            x = to_f32(static_cast<const T*>(a.q)[((int64_t)(b * (int64_t)g.T + m / G) * a.Hq + gkv * G + m % G) * a.dk + c]);
        qs[i] = x;
    }
    // the columns that a tile's rows do not fill
    for (int i = tid; i < kBufs * kKeys * (kp - a.dk); i += kThreads)
        ks_all[i / (kp - a.dk) * kp + a.dk + i % (kp - a.dk)] = 0.f;
    if (!latent && a.dv < vp)
        for (int i = tid; i < kBufs * kKeys * (vp - a.dv); i += kThreads)
            vs_all[i / (vp - a.dv) * vp + a.dv + i % (vp - a.dv)] = 0.f;
    __syncthreads();
    int k0 = INT32_MAX, k1 = 0, full0 = 0, full1 = INT32_MAX;
    for (int i = 0; i < R; ++i) {
        const int lo = lo_s[i], hi = hi_s[i];
        if (lo >= hi) continue;          // a row that sees nothing takes what it gets and writes zeros
        k0 = min(k0, lo);
        k1 = max(k1, hi);
        full0 = max(full0, lo);
        full1 = min(full1, hi);
    }
    // this split's share of them, in whole tiles
    if (k0 < k1) {
        const int64_t share = ((int64_t)(k1 - k0) + (int64_t)a.splits * kKeys - 1) / ((int64_t)a.splits * kKeys) * kKeys;
        const int64_t s0 = k0 + split * share, s1 = s0 + share;
        k0 = (int)min(s0, (int64_t)INT32_MAX);
        k1 = (int)min(s1, (int64_t)k1);
    }

    // a warp's rows are the same R / 4 in the scores, the softmax and the values: no barrier between them
    const int kg = tid % S::kKeyGroups;                               // scores
    const int r0 = tid / 32 * (R / 4) + tid % 32 / S::kKeyGroups;
    const int cg = tid % S::kColGroups, vg = tid / S::kColGroups;     // values
    constexpr int kPerRow = kThreads / R;                             // threads of a row's softmax
    const int srow = tid / kPerRow, sk = tid % kPerRow;
    uint64_t o[S::kRowsPer][2 * S::kCol4];                            // pairs of columns
#pragma unroll
    for (int i = 0; i < S::kRowsPer; ++i)
#pragma unroll
        for (int c = 0; c < 2 * S::kCol4; ++c) o[i][c] = 0ull;
    float m_run = -INFINITY, l_run = 0.f;
    const float cap = a.mods.softcap, inv_cap = cap > 0.f ? fminf(1.f / cap, FLT_MAX) : 0.f;   // (finite: 0 stays 0)

    // cache row of position j of the split, -1 past its end or outside the cache
    auto row_of = [&](int j) -> int64_t {
        if (j >= k1) return -1;
        const int64_t row = key_row(g, b, j);
        return row >= 0 && row < a.kv_rows ? row : -1;
    };
    // kAhead: four threads to a key, each every fourth 16-byte piece of its K and V rows (zeros for no row, and true)
    auto send = [&](int t0, int buf) {
        const int key = tid >> 2, sub = tid & 3;
        const int64_t row = t0 < k1 ? row_of(t0 + key) : -1;
        if (sub == 0) rows_all[buf * kKeys + key] = row;
        if (t0 < k1) {
            auto pieces = [&](const float* src, float* dst, int n) {
                const uint32_t d = sm100::smem_u32(dst);
                const int size = row >= 0 ? 16 : 0;
                for (int i = sub; i < n; i += 4)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + i * 16), "l"(src + i * 4), "r"(size)
                                 : "memory");
            };
            const int64_t at = row < 0 ? 0 : row;
            pieces(static_cast<const float*>(a.k) + at * a.k_stride + (int64_t)gkv * a.dk, ks_all + (buf * kKeys + key) * kp,
                   a.dk / 4);
            if (!latent)
                pieces(static_cast<const float*>(a.v) + at * a.v_stride + (int64_t)gkv * a.dv,
                       vs_all + (buf * kKeys + key) * vp, a.dv / 4);
        }
        return row < 0;
    };
    bool lost = false;                                                // this thread's key of the tile to come has no row
    if (kAhead) lost = send(k0, 0);
    int buf = 0;
    for (int t0 = k0; t0 < k1; t0 += kKeys) {
        float* ks = ks_all + buf * kKeys * kp;
        float* vs = latent ? ks : vs_all + buf * kKeys * vp;
        int64_t* rows_s = rows_all + buf * kKeys;
        bool bad;
        if constexpr (kAhead) {
            sm100::cp_async_wait_all();
            bad = __syncthreads_or(lost);       // this tile is there, and the last one is done with
            lost = send(t0 + kKeys, buf ^ 1);
            buf ^= 1;
        } else {
            __syncthreads();      // the last tile is done with
            if (tid < kKeys) rows_s[tid] = row_of(t0 + tid);
            bad = __syncthreads_or(tid < kKeys && rows_s[tid < kKeys ? tid : 0] < 0);
            // K and V rows, widened
            if (vec) {
                constexpr int E = 16 / (int)sizeof(T);
                const int wk = a.dk / E, wv = latent ? 0 : a.dv / E;
                const int total = kKeys * (wk + wv);
                constexpr int kBatch = 4;
                for (int e0 = tid; e0 < total; e0 += kThreads * kBatch) {
                    uint4 x[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int e = e0 + i * kThreads;
                        x[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (e < total) {
                            const bool isk = e < kKeys * wk;
                            const int ee = isk ? e : e - kKeys * wk, w = isk ? wk : wv;
                            const int64_t row = rows_s[ee / w];
                            if (row >= 0)
                                x[i] = *reinterpret_cast<const uint4*>(
                                    isk ? static_cast<const T*>(a.k) + row * a.k_stride + (int64_t)gkv * a.dk + ee % w * E
                                        : static_cast<const T*>(a.v) + row * a.v_stride + (int64_t)gkv * a.dv + ee % w * E);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int e = e0 + i * kThreads;
                        if (e < total) {
                            const bool isk = e < kKeys * wk;
                            const int ee = isk ? e : e - kKeys * wk, w = isk ? wk : wv;
                            float* d = isk ? ks + ee / w * kp + ee % w * E : vs + ee / w * vp + ee % w * E;
                            const T* p = reinterpret_cast<const T*>(&x[i]);
#pragma unroll
                            for (int j = 0; j < E; ++j) d[j] = to_f32(p[j]);
                        }
                    }
                }
            } else {
                for (int e = tid; e < kKeys * a.dk; e += kThreads) {
                    const int64_t row = rows_s[e / a.dk];
                    ks[e / a.dk * kp + e % a.dk] =
                        row >= 0 ? to_f32(static_cast<const T*>(a.k)[row * a.k_stride + (int64_t)gkv * a.dk + e % a.dk]) : 0.f;
                }
                if (!latent)
                    for (int e = tid; e < kKeys * a.dv; e += kThreads) {
                        const int64_t row = rows_s[e / a.dv];
                        vs[e / a.dv * vp + e % a.dv] =
                            row >= 0 ? to_f32(static_cast<const T*>(a.v)[row * a.v_stride + (int64_t)gkv * a.dv + e % a.dv])
                                     : 0.f;
                    }
            }
            __syncthreads();
        }
        // ---- scores
        const bool whole = !bad && t0 >= full0 && t0 + kKeys <= min(full1, k1);
        {
            uint64_t acc[4][S::kKeysPer];       // sums over even and over odd columns, packed
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < S::kKeysPer; ++j) acc[i][j] = 0ull;
            const float* qr = qs + r0 * kp;
            const float* kr = ks + kg * kp;
#pragma unroll 8
            for (int c = 0; c < kp - 4; c += 4) {
                ulonglong2 kk[S::kKeysPer], qq[4];
#pragma unroll
                for (int j = 0; j < S::kKeysPer; ++j)
                    kk[j] = *reinterpret_cast<const ulonglong2*>(kr + j * S::kKeyGroups * kp + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) qq[i] = *reinterpret_cast<const ulonglong2*>(qr + i * S::kRowStep * kp + c);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < S::kKeysPer; ++j)
                        acc[i][j] = fma2(qq[i].y, kk[j].y, fma2(qq[i].x, kk[j].x, acc[i][j]));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rr = r0 + i * S::kRowStep;
#pragma unroll
                for (int j = 0; j < S::kKeysPer; ++j) {
                    float even, odd;
                    unpair(acc[i][j], even, odd);
                    float x = (even + odd) * a.scale;
                    if (cap > 0.f) x = cap * tanhf(x * inv_cap);
                    const int kl = kg + j * S::kKeyGroups;
                    if (a.mods.slopes) x -= slope_s[rr] * fabsf((float)((int64_t)pos_s[rr] - (t0 + kl)));
                    ss[kl * (R + 4) + rr] = x;
                }
            }
        }
        __syncwarp();
        // ---- softmax: kPerRow threads of a warp per row; a masked key's weight is marked by -1
        {
            const int lo = lo_s[srow], hi = hi_s[srow];
            const bool none = lo >= hi;
            float mt = -INFINITY;
            uint32_t seen = 0u;
#pragma unroll
            for (int j = 0; j < kKeys / kPerRow; ++j) {
                const int kl = sk + j * kPerRow;
                const int key = t0 + kl;
                const bool v = whole ? !none : (key >= lo && key < hi && key < k1 && rows_s[kl] >= 0);
                if (v) {
                    seen |= 1u << j;
                    mt = fmaxf(mt, ss[kl * (R + 4) + srow]);
                }
            }
#pragma unroll
            for (int off = 1; off < kPerRow; off <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
            if (bad) {      // a key outside the cache counts where a row sees it
                for (int kl = sk; kl < kKeys; kl += kPerRow)
                    if (rows_s[kl] < 0 && t0 + kl >= lo && t0 + kl < min(hi, k1)) flag(g.status, IDX_ERR_DEVICE_BOUNDS);
            }
            const float m_new = fmaxf(m_run, mt);
            const float m_ref = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = m_run == m_new ? 1.f : expf(m_run - m_ref);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < kKeys / kPerRow; ++j) {
                float* p = ss + (sk + j * kPerRow) * (R + 4) + srow;
                if ((seen >> j) & 1u) {
                    const float w = expf(*p - m_ref);
                    *p = w;
                    sum += w;
                } else {
                    *p = -1.f;
                }
            }
#pragma unroll
            for (int off = 1; off < kPerRow; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l_run = l_run * alpha + sum;
            m_run = m_new;
            if (sk == 0) alpha_s[srow] = alpha;
        }
        __syncwarp();
        // ---- values
        bool scaled = false;
#pragma unroll
        for (int i = 0; i < S::kRowsPer; ++i) scaled |= alpha_s[vg * S::kRowsPer + i] != 1.f;
        if (scaled) {
#pragma unroll
            for (int i = 0; i < S::kRowsPer; ++i) {
                const float al = alpha_s[vg * S::kRowsPer + i];
#pragma unroll
                for (int c = 0; c < 2 * S::kCol4; ++c) o[i][c] = mul2(o[i][c], pair(al, al));
            }
        }
        const int n_keys = min(kKeys, k1 - t0);
        auto values = [&](auto masked) {
#pragma unroll 8
            for (int kl = 0; kl < n_keys; ++kl) {
                float p[S::kRowsPer];
#pragma unroll
                for (int i = 0; i < S::kRowsPer; i += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(ss + kl * (R + 4) + vg * S::kRowsPer + i);
                    p[i] = x.x;
                    p[i + 1] = x.y;
                    p[i + 2] = x.z;
                    p[i + 3] = x.w;
                }
#pragma unroll
                for (int c = 0; c < S::kCol4; ++c) {
                    const int col = 4 * cg + 4 * S::kColGroups * c;
                    if (col >= a.dv) continue;
                    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(vs + kl * vp + col);
#pragma unroll
                    for (int i = 0; i < S::kRowsPer; ++i) {
                        if (decltype(masked)::value && p[i] < 0.f) continue;
                        const uint64_t pp = pair(p[i], p[i]);
                        o[i][2 * c] = fma2(pp, x.x, o[i][2 * c]);
                        o[i][2 * c + 1] = fma2(pp, x.y, o[i][2 * c + 1]);
                    }
                }
            }
        };
        if (whole)
            values(std::false_type{});
        else
            values(std::true_type{});
    }

    if (kAhead) sm100::cp_async_wait_all();
    // ---- output: m and l per row through shared memory
    const bool merge = a.splits > 1 && !a.part_o;       // the splits are the CTAs of a cluster
    float* m_s = slope_s;
    float* l_s = alpha_s;
    __syncthreads();
    if (sk == 0) {
        const bool none = lo_s[srow] >= hi_s[srow];
        const float l = none ? 0.f : l_run;
        l_s[srow] = l;
        m_s[srow] = m_run;
        const int64_t m = m0 + srow;
        if (m < m_end && !merge) {
            const int64_t rh = ((int64_t)b * g.T + m / G) * a.Hq + gkv * G + m % G;
            if (a.splits > 1) {
                a.part_ml[(rh * a.splits + split) * 2] = m_run;
                a.part_ml[(rh * a.splits + split) * 2 + 1] = l;
            } else if (a.lse) {
                a.lse[rh] = l == 0.f ? -INFINITY : m_run + logf(l);
            }
        }
    }
    __syncthreads();
    float* o_s = qs;                                    // [R][dv], merge: over what nobody reads any more
#pragma unroll
    for (int i = 0; i < S::kRowsPer; ++i) {
        const int rr = vg * S::kRowsPer + i;
        const int64_t m = m0 + rr;
        if (m >= m_end) continue;
        const int64_t rh = ((int64_t)b * g.T + m / G) * a.Hq + gkv * G + m % G;
        const float l = l_s[rr];
        const float inv = a.splits > 1 ? 1.f : 1.f / l;
#pragma unroll
        for (int c = 0; c < S::kCol4; ++c) {
            float oc[4];
            unpair(o[i][2 * c], oc[0], oc[1]);
            unpair(o[i][2 * c + 1], oc[2], oc[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = 4 * cg + 4 * S::kColGroups * c + e;
                if (col >= a.dv) continue;
                const float x = l == 0.f ? 0.f : oc[e] * inv;
                if (merge)
                    o_s[rr * a.dv + col] = x;
                else if (a.splits > 1)
                    a.part_o[(rh * a.splits + split) * a.dv + col] = x;
                else
                    static_cast<T*>(a.out)[rh * a.dv + col] = from_f32<T>(x);
            }
        }
    }
    if (merge) {
        // each CTA merges its share of the elements, in the order of the splits
        sm100::cluster_sync();
        const int rows = (int)min((int64_t)R, m_end - m0);
        for (int e = split * kThreads + tid; e < rows * a.dv; e += a.splits * kThreads) {
            const int rr = e / a.dv, col = e - rr * a.dv;
            float mx[kDenseCluster], lx[kDenseCluster], ox[kDenseCluster];
#pragma unroll
            for (int s = 0; s < kDenseCluster; ++s) {
                const int from = s < a.splits ? s : 0;
                mx[s] = *sm100::of_cta(m_s + rr, from);
                lx[s] = s < a.splits ? *sm100::of_cta(l_s + rr, from) : 0.f;
                ox[s] = *sm100::of_cta(o_s + e, from);
            }
            float M = -INFINITY, den = 0.f, acc = 0.f;
#pragma unroll
            for (int s = 0; s < kDenseCluster; ++s)
                if (lx[s] != 0.f) M = fmaxf(M, mx[s]);
#pragma unroll
            for (int s = 0; s < kDenseCluster; ++s)
                if (lx[s] != 0.f) {
                    const float w = expf(mx[s] - M);
                    den = fmaf(w, lx[s], den);
                    acc = fmaf(w, ox[s], acc);
                }
            const int64_t m = m0 + rr;
            const int64_t rh = ((int64_t)b * g.T + m / G) * a.Hq + gkv * G + m % G;
            static_cast<T*>(a.out)[rh * a.dv + col] = from_f32<T>(den == 0.f ? 0.f : acc / den);
            if (a.lse && col == 0) a.lse[rh] = den == 0.f ? -INFINITY : M + logf(den);
        }
        sm100::cluster_sync();      // no CTA leaves while another reads its memory
    }
}

// one warp per (row, head): out = sum_s e^(m_s - M) o_s / sum_s e^(m_s - M) l_s.  Lane s holds the weights of
// splits s, s + 32, ...; a lane sums V consecutive columns, the splits' loads issued kBatch at a time.
template <typename T, int V>
__global__ void __launch_bounds__(128) dense_combine_kernel(DenseArgs a, int64_t n) {
    constexpr int kSplits = kDenseMaxSplits / 32, kBatch = 8;
    pdl_wait();
    const int64_t rh = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (rh >= n) return;
    const float* ml = a.part_ml + rh * a.splits * 2;
    float m[kSplits], l[kSplits], M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSplits; ++i) {
        const int s = lane + 32 * i;
        m[i] = s < a.splits ? ml[2 * s] : 0.f;
        l[i] = s < a.splits ? ml[2 * s + 1] : 0.f;
        if (l[i] != 0.f) M = fmaxf(M, m[i]);      // (a split without keys has l = 0; a NaN counts)
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float den = 0.f;
#pragma unroll
    for (int i = 0; i < kSplits; ++i) {
        m[i] = l[i] != 0.f ? expf(m[i] - M) : 0.f;
        den += m[i] * l[i];
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
    if (a.lse && lane == 0) a.lse[rh] = den == 0.f ? -INFINITY : M + logf(den);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    for (int c0 = 0; c0 < a.dv; c0 += 32 * V) {
        const int c = c0 + lane * V;
        float acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll
        for (int i = 0; i < kSplits; ++i) {
            for (int s0 = 0; s0 < 32 && 32 * i + s0 < a.splits; s0 += kBatch) {
                float x[kBatch][V];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
#pragma unroll
                    for (int v = 0; v < V; ++v) x[k][v] = 0.f;
                    const int s = 32 * i + s0 + k;
                    if (s < a.splits && c < a.dv) {
                        const float* p = a.part_o + (rh * a.splits + s) * a.dv + c;
                        if constexpr (V == 4) {
                            const float4 y = *reinterpret_cast<const float4*>(p);
                            x[k][0] = y.x;
                            x[k][1] = y.y;
                            x[k][2] = y.z;
                            x[k][3] = y.w;
                        } else {
                            x[k][0] = *p;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const float w = __shfl_sync(0xffffffffu, m[i], s0 + k);
                    // (a split without keys wrote zeros)
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[v] = fmaf(w, x[k][v], acc[v]);
                }
            }
        }
        if (c < a.dv) {
            T* o = static_cast<T*>(a.out) + rh * a.dv + c;
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = from_f32<T>(acc[v] * inv);
        }
    }
}

// rows of a CTA's tile: 64 when the sequence's packed rows fill more than one tile of 16, the values are at most 128 wide
// (the wider output block needs the registers) and the keys at most 528 (231,680 bytes of shared memory with values of
// 128 beside them; 529 columns take 233,216, more than the 232,448 that a CTA may have)
int tile_rows(int64_t packed, int dk, int dv) { return dv <= 128 && dk <= 528 && packed > 16 ? 64 : 16; }

template <typename T>
cudaError_t run(const DenseArgs& a, const Geom& g, cudaStream_t st) {
    const int64_t packed = (int64_t)g.T * (a.Hq / a.Hkv);
    const int R = tile_rows(packed, a.dk, a.dv);
    const int64_t tiles = (packed + R - 1) / R;
    const int64_t grid = (int64_t)g.B * a.Hkv * tiles * a.splits;
    if (grid > INT32_MAX || tiles > INT32_MAX) return cudaErrorNotSupported;
    const uint64_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                         (uint64_t)a.k_stride * sizeof(T) | (a.v ? (uint64_t)a.v_stride * sizeof(T) : 0) |
                         (uint64_t)a.dk * sizeof(T) | (a.v ? (uint64_t)a.dv * sizeof(T) : 0);
    const bool vec = all % 16 == 0;
    auto go = [&](auto kern, int dvp, int bufs) {
        const size_t sm = smem_bytes(R, dvp, a.dk, a.dv, !a.v, bufs);
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
        if (e != cudaSuccess) return e;
        return launch_pdl_cluster(kern, dim3((unsigned)grid), dim3(kThreads), sm, st,
                                  a.splits > 1 && !a.part_o ? a.splits : 1, a, g, (int)tiles, vec);
    };
    if constexpr (sizeof(T) == 4) {
        // a tile ahead where two CTAs fit an SM with it (wider rows would be alone there)
        const int dvp = R == 64 && a.dv <= 64 ? 64 : a.dv <= 128 ? 128 : 512;
        if (vec && smem_bytes(R, dvp, a.dk, a.dv, !a.v, 2) <= 113 * 1024) {
            if (R == 64)
                return dvp == 64 ? go(dense_generic_kernel<T, 64, 64, true>, 64, 2) : go(dense_generic_kernel<T, 64, 128, true>, 128, 2);
            if (dvp == 128) return go(dense_generic_kernel<T, 16, 128, true>, 128, 2);
        }
    }
    if (R == 64)
        return a.dv <= 64 ? go(dense_generic_kernel<T, 64, 64, false>, 64, 1) : go(dense_generic_kernel<T, 64, 128, false>, 128, 1);
    return a.dv <= 128 ? go(dense_generic_kernel<T, 16, 128, false>, 128, 1) : go(dense_generic_kernel<T, 16, 512, false>, 512, 1);
}

}  // namespace

// enough CTAs to cover the SMs four times, at least a tile of keys each: a tile takes about 4 us whatever it holds
// (256 keys for one token of four f32 heads: 19.7 us in two splits, 10.5 in eight)
int dense_generic_splits(int64_t n_seq, int64_t n_q, int64_t max_n_kv, int Hq, int Hkv, int dk, int dv) {
    const int64_t packed = n_q * (Hq / Hkv);
    const int R = tile_rows(packed, dk, dv);
    const int64_t units = n_seq * Hkv * ((packed + R - 1) / R);
    int sms = sm_count();
    if (sms < 2) sms = 152;
    if (units < 1) return 1;
    int64_t s = 4 * (int64_t)sms / units;
    const int64_t by_keys = (max_n_kv + kKeys - 1) / kKeys;
    if (s > by_keys) s = by_keys;
    if (s > kDenseMaxSplits) s = kDenseMaxSplits;
    return s < 1 ? 1 : (int)s;
}

cudaError_t launch_dense_generic(const DenseArgs& a, int dtype, const Geom& g, cudaStream_t st) {
    switch (dtype) {
        case IDX_F16: return run<__half>(a, g, st);
        case IDX_BF16: return run<__nv_bfloat16>(a, g, st);
        default: return run<float>(a, g, st);
    }
}

template <typename T>
static cudaError_t combine(const DenseArgs& a, int64_t n, cudaStream_t st) {
    const dim3 grid((unsigned)((n + 3) / 4));
    return a.dv % 4 == 0 ? launch_pdl(dense_combine_kernel<T, 4>, grid, dim3(128), 0, st, a, n)
                         : launch_pdl(dense_combine_kernel<T, 1>, grid, dim3(128), 0, st, a, n);
}

cudaError_t launch_dense_combine(const DenseArgs& a, int dtype, int64_t n_rows, cudaStream_t st) {
    const int64_t n = n_rows * a.Hq;
    switch (dtype) {
        case IDX_F16: return combine<__half>(a, n, st);
        case IDX_BF16: return combine<__nv_bfloat16>(a, n, st);
        default: return combine<float>(a, n, st);
    }
}

}  // namespace lidx
