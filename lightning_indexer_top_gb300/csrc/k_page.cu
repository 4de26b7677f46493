// The pages of paged caches: copying listed pages, a step's update of a page
// table (free, truncate, fork, grow) and compaction.
//
// A page is owned by the table rows that name it, so the plan of an update or a
// compaction starts from a bitmap of the named pages; ranks in the bitmap (a
// prefix sum of its words' zero counts) give the k-th free page, so the result
// depends on nothing but the inputs.  The plan runs on one cluster; the page
// contents then move in a second launch over all SMs.
#include "lidx_internal.cuh"
#include "sm100_ptx.cuh"

namespace lidx {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 128;
constexpr int kSegBytes = 16384;   // bytes of a page that a CTA copies at a time

struct Caches {
    idx_page_cache c[IDX_MAX_PAGE_CACHES];
    int32_t vec[IDX_MAX_PAGE_CACHES];    // widest load that pointer, stride and payload allow (bytes)
    int32_t segs[IDX_MAX_PAGE_CACHES];   // kSegBytes pieces of a page's payload
    int32_t n;
    int32_t segs_total;
    int32_t page_size;
};

// the pages that a plan hands to the copy kernel
struct Moves {
    const int32_t* src;
    const int32_t* dst;
    const int32_t* rows;    // rows of each page that move, or NULL: all
    const int32_t* n_dev;   // their number on the device, or NULL: n
    int32_t n;
};

template <typename V>
__device__ __forceinline__ void copy_piece(const uint8_t* src, uint8_t* dst, int64_t row_bytes, int64_t stride,
                                           int o0, int o1) {
    constexpr int kBatch = 8;
    constexpr int S = (int)sizeof(V);
    if (row_bytes == stride) {
        const V* s = reinterpret_cast<const V*>(src + o0) + threadIdx.x;
        V* d = reinterpret_cast<V*>(dst + o0) + threadIdx.x;
        const int n = (o1 - o0) / S - (int)threadIdx.x;     // this thread's share ends n elements on
        int i0 = 0;
        for (; i0 + (kBatch - 1) * kCopyThreads < n; i0 += kBatch * kCopyThreads) {
            V v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] = __ldcs(s + i0 + i * kCopyThreads);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) __stcs(d + i0 + i * kCopyThreads, v[i]);
        }
        for (; i0 < n; i0 += kCopyThreads) __stcs(d + i0, __ldcs(s + i0));
    } else {
        // rows with bytes between them that are not the cache's
        for (int o = o0 + (int)threadIdx.x * S; o < o1; o += kCopyThreads * S) {
            const int64_t at = o / row_bytes * stride + o % row_bytes;
            __stcs(reinterpret_cast<V*>(dst + at), __ldcs(reinterpret_cast<const V*>(src + at)));
        }
    }
}

// a stream of reads and writes: HBM is what bounds it
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(Caches cs, Moves m, int32_t n_pages, int* status) {
    pdl_wait();
    const int64_t n = m.n_dev ? *m.n_dev : m.n;
    for (int64_t w = blockIdx.x; w < n * cs.segs_total; w += gridDim.x) {
        const int64_t item = w / cs.segs_total;
        int seg = (int)(w - item * cs.segs_total);
        const int32_t s = m.src[item], d = m.dst[item];
        if (s < 0 || d < 0 || s == d) continue;
        if (s >= n_pages || d >= n_pages) {
            if (seg == 0 && threadIdx.x == 0) flag(status, IDX_ERR_DEVICE_BOUNDS);
            continue;
        }
        int c = 0;
        while (seg >= cs.segs[c]) seg -= cs.segs[c++];
        const int64_t stride = cs.c[c].row_stride_bytes, rb = cs.c[c].row_bytes;
        // (a page's payload is below 2^31 bytes)
        const int end = (int)((int64_t)(m.rows ? m.rows[item] : cs.page_size) * rb);
        const int o0 = seg * kSegBytes;
        const int o1 = min(o0 + kSegBytes, end);
        if (o0 >= o1) continue;
        const uint8_t* sp = static_cast<const uint8_t*>(cs.c[c].data) + (int64_t)s * cs.page_size * stride;
        uint8_t* dp = static_cast<uint8_t*>(cs.c[c].data) + (int64_t)d * cs.page_size * stride;
        switch (cs.vec[c]) {
            case 16: copy_piece<uint4>(sp, dp, rb, stride, o0, o1); break;
            case 8: copy_piece<uint2>(sp, dp, rb, stride, o0, o1); break;
            case 4: copy_piece<uint32_t>(sp, dp, rb, stride, o0, o1); break;
            case 2: copy_piece<uint16_t>(sp, dp, rb, stride, o0, o1); break;
            default: copy_piece<uint8_t>(sp, dp, rb, stride, o0, o1); break;
        }
    }
}

// ---------------------------------------------------------------- the plan: one cluster of kCl CTAs
//
// Each CTA holds a slice of the bitmap in shared memory (in the workspace when it
// is too long), marks pages in all of them, and walks its share of the rows.  A
// step ends with a cluster barrier, whose release and acquire also cover the
// global arrays.  (One CTA with the bitmap in global memory took 50 us for 256
// rows of 256 pages, and 248 us to plan a compaction of 32768 pages; eight with the
// bitmap in theirs 23 us, the copies and both launches included, and about 20.)
constexpr int kCl = 8;
constexpr int kWarps = kPlanThreads / 32;
constexpr int kSliceWords = 24 * 1024;     // words of a slice up to which it is kept (twice) in shared memory

struct Plan {
    int cnt[4][kCl];       // counts that the CTAs tell one another
    int scan[32];
};

__device__ __forceinline__ uint32_t cta_rank() { return sm100::cluster_ctarank(); }

// the exclusive prefix sum of x over the CTA's threads; *total gets the sum
__device__ __forceinline__ int block_scan(Plan& s, int x, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();   // the last call's sums have been read
    if (lane == 31) s.scan[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
    const int v = lane < kWarps ? s.scan[lane] : 0;
    before = lane < warp ? v : 0;
    all = v;
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    *total = all;
    return inc - x + before;
}

// tells every CTA x of this one in cnt[k]; after the next cluster barrier, the sum before this CTA and in all
__device__ __forceinline__ void tell(Plan& s, int k, int x) {
    if (threadIdx.x < kCl) sm100::of_cta(&s.cnt[k][0], threadIdx.x)[cta_rank()] = x;
}
__device__ __forceinline__ int told(const Plan& s, int k, int* total) {
    int before = 0, all = 0;
    for (int i = 0; i < kCl; ++i) {
        if (i < (int)cta_rank()) before += s.cnt[k][i];
        all += s.cnt[k][i];
    }
    *total = all;
    return before;
}

// the bitmap of the pages: word w is word w - rank * slice of CTA w / slice
struct Bitmap {
    uint32_t* mine;        // this CTA's slice
    uint32_t* global;      // the whole bitmap in the workspace, or NULL: slices in shared memory
    int slice;             // words per slice
    int words;

    __device__ __forceinline__ uint32_t* word(int w) const {
        return global ? global + w : sm100::of_cta(mine, (uint32_t)(w / slice)) + w % slice;
    }
    __device__ __forceinline__ void set(int32_t p) const { atomicOr(word(p >> 5), 1u << (p & 31)); }
    __device__ __forceinline__ bool get(int32_t p) const {
        return (*(volatile uint32_t*)word(p >> 5) >> (p & 31)) & 1u;
    }
    // words of this CTA's slice
    __device__ __forceinline__ int n_mine() const {
        const int left = words - (int)cta_rank() * slice;
        return left < 0 ? 0 : left < slice ? left : slice;
    }
};

__device__ __forceinline__ Bitmap make_bitmap(uint32_t* ws, uint32_t* smem, int32_t n_pages) {
    Bitmap m;
    m.words = (int)(((int64_t)n_pages + 31) / 32);
    m.slice = (m.words + kCl - 1) / kCl;
    if (m.slice < 1) m.slice = 1;
    m.global = m.slice > kSliceWords ? ws : nullptr;
    m.mine = m.global ? ws + (int64_t)cta_rank() * m.slice : smem;
    return m;
}

// bits of word w that are numbers below n
__device__ __forceinline__ uint32_t page_bits(int64_t w, int32_t n) {
    const int64_t left = (int64_t)n - w * 32;
    return left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
}

__device__ __forceinline__ uint32_t held_bits(const uint8_t* held, int64_t w, int32_t n_pages) {
    if (!held) return 0u;
    uint32_t x = 0u;
    const int64_t p0 = w * 32;
    if (p0 + 32 <= n_pages && !(reinterpret_cast<uintptr_t>(held) & 15u)) {
        const uint4 a = reinterpret_cast<const uint4*>(held + p0)[0], b = reinterpret_cast<const uint4*>(held + p0)[1];
        const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 32; ++i) x |= ((v[i >> 2] >> (8 * (i & 3))) & 0xffu ? 1u : 0u) << i;
    } else {
        for (int i = 0; i < 32 && p0 + i < n_pages; ++i) x |= (held[p0 + i] ? 1u : 0u) << i;
    }
    return x;
}

struct UpdateArgs {
    const int32_t* table;
    int64_t stride;
    int32_t cols, n_old;
    const int32_t *parent, *keep, *len;
    int32_t n_seq, ps, n_pages;
    const uint8_t* held;
    int32_t* out;
    int64_t out_stride;
    int32_t out_cols;
    int32_t* n_free;
    uint32_t* bm;          // [words]
    int32_t* list;         // [n_pages] who wants a page kept in part, then the free pages in order
    int32_t* offset;       // [n_seq] first new page of the row in the list
    int32_t *src, *dst, *rows;   // [n_seq] the copies (src -1: none)
    int* status;
};

// calls f(entry, index) for the first n entries of a row, the lanes of a warp together
template <typename F>
__device__ __forceinline__ void each_entry(const int32_t* row, int n, F f) {
    constexpr int kBatch = 8;
    const int lane = threadIdx.x & 31;
    for (int i0 = lane; i0 < n; i0 += 32 * kBatch) {
        int32_t v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) v[k] = i0 + 32 * k < n ? row[i0 + 32 * k] : 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (i0 + 32 * k < n) f(v[k], i0 + 32 * k);
    }
}

__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kPlanThreads) page_update_kernel(UpdateArgs a) {
    extern __shared__ uint32_t slice_s[];
    __shared__ Plan s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)cta_rank();
    const Bitmap bm = make_bitmap(a.bm, slice_s, a.n_pages);
    const int gtid = rank * kPlanThreads + tid;            // of the cluster: rows are dealt out by thread ...
    const int gwarp = rank * kWarps + warp;                // ... or by warp
    constexpr int kAll = kCl * kPlanThreads, kAllWarps = kCl * kWarps;
    sm100::cluster_arrive();        // this CTA has started: from the wait on, the others may write to its memory
    pdl_wait();
    // ---- the requests; the held pages.  Nothing is copied unless the plan says so.
    bool bad = false;
    for (int b = gtid; b < a.n_seq; b += kAll) {
        const int32_t p = a.parent[b], k = a.keep[b], n = a.len[b];
        bad |= p < -1 || p >= a.n_old || k < 0 || n < k || (p < 0 && k > 0) ||
               (int64_t)k > (int64_t)a.cols * a.ps || (int64_t)n > (int64_t)a.out_cols * a.ps;
        a.src[b] = -1;
    }
    for (int w = tid; w < bm.n_mine(); w += kPlanThreads)
        bm.mine[w] = held_bits(a.held, (int64_t)rank * bm.slice + w, a.n_pages);
    bad = __syncthreads_or(bad);
    sm100::cluster_wait();
    tell(s, 0, bad ? 1 : 0);
    sm100::cluster_sync();
    int any;
    told(s, 0, &any);
    auto impossible = [&] {
        for (int b = gtid; b < a.n_seq; b += kAll) a.src[b] = -1;
        if (gtid == 0) {
            *a.n_free = INT32_MIN;
            flag(a.status, IDX_ERR_DEVICE_BOUNDS);
        }
    };
    if (any) {
        impossible();
        return;
    }
    // ---- pages kept whole
    for (int b = gwarp; b < a.n_seq; b += kAllWarps) {
        const int whole = a.keep[b] / a.ps, part = a.keep[b] % a.ps;
        const int n = whole + (part ? 1 : 0);
        if (n == 0) continue;
        each_entry(a.table + (int64_t)a.parent[b] * a.stride, n, [&](int32_t p, int i) {
            if (p < 0 || p >= a.n_pages)
                bad = true;
            else if (i < whole)
                bm.set(p);
            else {
                a.src[b] = p;
                a.list[p] = INT32_MAX;      // wanted by nobody yet (the same value from every row that names it)
            }
        });
    }
    bad = __syncthreads_or(bad);
    tell(s, 1, bad ? 1 : 0);
    sm100::cluster_sync();
    told(s, 1, &any);
    if (any) {
        impossible();
        return;
    }
    // ---- the pages kept in part: the first row that wants one has it, unless it is kept whole or held
    for (int b = gtid; b < a.n_seq; b += kAll) {
        const int32_t p = a.src[b];
        if (p >= 0 && !bm.get(p)) atomicMin(a.list + p, b);
    }
    sm100::cluster_sync();
    for (int b = gtid; b < a.n_seq; b += kAll) {
        const int32_t p = a.src[b];
        const bool stays = p >= 0 && *(volatile int32_t*)(a.list + p) == b;
        a.rows[b] = p < 0 || stays ? 0 : a.keep[b] % a.ps;   // rows to copy
    }
    sm100::cluster_sync();      // (every bit has been read)
    for (int b = gtid; b < a.n_seq; b += kAll)
        if (a.src[b] >= 0 && a.rows[b] == 0) bm.set(a.src[b]);
    // ---- new pages of each row, in order (every CTA adds up all of them)
    int need = 0;
    for (int b0 = 0; b0 < a.n_seq; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int x = 0;
        if (b < a.n_seq) {
            const int pages = (int)(((int64_t)a.len[b] + a.ps - 1) / a.ps);
            x = pages - a.keep[b] / a.ps - (a.src[b] >= 0 && a.rows[b] == 0 ? 1 : 0);
        }
        int total;
        const int at = block_scan(s, x, &total);
        if (b < a.n_seq && b % kAllWarps / kWarps == rank) a.offset[b] = need + at;   // (its own rows)
        need += total;
    }
    sm100::cluster_sync();
    // ---- the free pages, in order, as many as are needed
    int zeros = 0;
    for (int w = tid; w < bm.n_mine(); w += kPlanThreads)
        zeros += __popc(~bm.mine[w] & page_bits((int64_t)rank * bm.slice + w, a.n_pages));
    int mine;
    block_scan(s, zeros, &mine);
    tell(s, 2, mine);
    sm100::cluster_sync();
    int n_free;
    int at0 = told(s, 2, &n_free);
    if (gtid == 0) *a.n_free = n_free - need;
    if (n_free < need) {
        for (int b = gtid; b < a.n_seq; b += kAll) a.src[b] = -1;
        return;
    }
    for (int w0 = 0; w0 < bm.n_mine() && at0 < need; w0 += kPlanThreads) {
        const int w = w0 + tid;
        const int64_t gw = (int64_t)rank * bm.slice + w;
        uint32_t z = w < bm.n_mine() ? ~bm.mine[w] & page_bits(gw, a.n_pages) : 0u;
        int total;
        int at = at0 + block_scan(s, __popc(z), &total);
        for (; z && at < need; z &= z - 1, ++at) a.list[at] = (int32_t)(gw * 32) + __ffs((int)z) - 1;
        at0 += total;
    }
    sm100::cluster_sync();
    // ---- the new rows
    for (int b = gwarp; b < a.n_seq; b += kAllWarps) {
        const int whole = a.keep[b] / a.ps;
        const int pages = (int)(((int64_t)a.len[b] + a.ps - 1) / a.ps);
        const int32_t last = a.src[b];
        const bool stays = last >= 0 && a.rows[b] == 0;
        const int kept = whole + (stays ? 1 : 0);
        const int32_t* row = a.table + (int64_t)(kept ? a.parent[b] : 0) * a.stride;
        const int32_t* list = a.list + a.offset[b] - kept;
        int32_t* out = a.out + (int64_t)b * a.out_stride;
        each_entry(row, kept, [&](int32_t p, int i) { out[i] = p; });
        for (int i = kept + lane; i < a.out_cols; i += 32) out[i] = i < pages ? list[i] : -1;
        __syncwarp();
        if (lane == 0) {
            if (stays)
                a.src[b] = -1;
            else if (last >= 0)
                a.dst[b] = list[whole];
        }
    }
}

struct CompactArgs {
    const int32_t* table;
    int64_t stride;
    int32_t cols, n_seq;
    const int32_t* len;
    int32_t ps, n_pages;
    const uint8_t* held;
    int32_t* out;
    int64_t out_stride;
    int32_t *n_used, *remap;
    uint32_t *bm, *moving;   // [words] used or held; moving (unused where both fit shared memory)
    int32_t *src, *dst; // [n_pages / 2 + 1] the moves
    int32_t* n_moves;
    int* status;
};

__device__ __forceinline__ int live_pages(const CompactArgs& a, int b) {
    int64_t n = a.len[b];
    const int64_t most = (int64_t)a.cols * a.ps;
    if (n < 0 || n > most) {
        flag(a.status, IDX_ERR_DEVICE_BOUNDS);
        n = n < 0 ? 0 : most;
    }
    return (int)((n + a.ps - 1) / a.ps);
}

__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kPlanThreads) page_compact_kernel(CompactArgs a) {
    extern __shared__ uint32_t slice_s[];
    __shared__ Plan s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)cta_rank();
    const Bitmap bm = make_bitmap(a.bm, slice_s, a.n_pages);
    const int gwarp = rank * kWarps + warp;
    constexpr int kAllWarps = kCl * kWarps;
    const int64_t w_base = (int64_t)rank * bm.slice;
    pdl_wait();
    for (int w = tid; w < bm.n_mine(); w += kPlanThreads) bm.mine[w] = held_bits(a.held, w_base + w, a.n_pages);
    sm100::cluster_sync();
    for (int b = gwarp; b < a.n_seq; b += kAllWarps)
        each_entry(a.table + (int64_t)b * a.stride, live_pages(a, b), [&](int32_t p, int) {
            if (p >= 0 && p < a.n_pages)
                bm.set(p);
            else
                flag(a.status, IDX_ERR_DEVICE_BOUNDS);
        });
    sm100::cluster_sync();
    int x = 0, total;
    for (int w = tid; w < bm.n_mine(); w += kPlanThreads) x += __popc(bm.mine[w]);
    block_scan(s, x, &total);
    tell(s, 0, total);
    sm100::cluster_sync();
    int n_used;
    told(s, 0, &n_used);
    // the moving pages (used, not held, numbered n_used or higher) and the free numbers below, in order
    uint32_t* moving = bm.global ? a.moving + w_base : slice_s + bm.slice;
    auto holes = [&](int w) { return ~bm.mine[w] & page_bits(w_base + w, n_used); };
    int y = 0;
    x = 0;
    for (int w = tid; w < bm.n_mine(); w += kPlanThreads) {     // (each word by the same thread from here on)
        const int64_t gw = w_base + w;
        moving[w] = bm.mine[w] & ~held_bits(a.held, gw, a.n_pages) & ~page_bits(gw, n_used);
        x += __popc(moving[w]);
        y += __popc(holes(w));
    }
    block_scan(s, x, &total);
    tell(s, 1, total);
    block_scan(s, y, &total);
    tell(s, 2, total);
    sm100::cluster_sync();
    int n_moves, n_holes;
    const int mv0 = told(s, 1, &n_moves);
    int ho0 = told(s, 2, &n_holes);
    int at0 = mv0;
    for (int w0 = 0; w0 < bm.n_mine(); w0 += kPlanThreads) {
        const int w = w0 + tid;
        const bool in = w < bm.n_mine();
        uint32_t m = in ? moving[w] : 0u;
        int at = at0 + block_scan(s, __popc(m), &total);
        at0 += total;
        for (; m; m &= m - 1, ++at) a.src[at] = (int32_t)((w_base + w) * 32) + __ffs((int)m) - 1;
        m = in ? holes(w) : 0u;
        at = ho0 + block_scan(s, __popc(m), &total);
        ho0 += total;
        for (; m; m &= m - 1, ++at) a.dst[at] = (int32_t)((w_base + w) * 32) + __ffs((int)m) - 1;
    }
    if (rank == 0 && tid == 0) {
        *a.n_used = n_used;
        *a.n_moves = n_moves;
    }
    sm100::cluster_sync();
    // the new number of every page of the slice: a thread per word, then the warp walks its 32 words together
    at0 = mv0;
    for (int w0 = 0; w0 < bm.n_mine(); w0 += kPlanThreads) {
        const int w = w0 + tid;
        const uint32_t m = w < bm.n_mine() ? moving[w] : 0u;
        const int at = at0 + block_scan(s, __popc(m), &total);
        at0 += total;
        const int64_t p0 = (w_base + w0 + warp * 32) * 32 + lane;
        const int n_words = min(32, bm.n_mine() - w0 - warp * 32);
        constexpr int kBatch = 8;
        for (int k0 = 0; k0 < n_words; k0 += kBatch) {
            int32_t to[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t mk = __shfl_sync(0xffffffffu, m, k0 + k);
                const int ak = __shfl_sync(0xffffffffu, at, k0 + k);
                const int64_t p = p0 + (int64_t)(k0 + k) * 32;
                to[k] = (mk >> lane) & 1u ? a.dst[ak + __popc(mk & ((1u << lane) - 1u))] : (int32_t)p;
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int64_t p = p0 + (int64_t)(k0 + k) * 32;
                if (k0 + k < n_words && p < a.n_pages) a.remap[p] = to[k];
            }
        }
    }
    sm100::cluster_sync();
    for (int b = gwarp; b < a.n_seq; b += kAllWarps) {
        const int n = live_pages(a, b);
        int32_t* out = a.out + (int64_t)b * a.out_stride;
        each_entry(a.table + (int64_t)b * a.stride, n, [&](int32_t p, int i) {
            out[i] = p >= 0 && p < a.n_pages ? *(volatile int32_t*)(a.remap + p) : -1;
        });
        for (int i = n + lane; i < a.cols; i += 32) out[i] = -1;
    }
}

size_t align16(size_t x) { return (x + 15) & ~size_t(15); }

size_t bitmap_bytes(int64_t n_pages) {
    const size_t slice = ((size_t)(n_pages + 31) / 32 + kCl - 1) / kCl;
    return align16((slice ? slice : 1) * kCl * 4);
}

// launches a plan: the bitmap's slices in shared memory where they fit
template <typename Args>
cudaError_t launch_plan(void (*kern)(Args), const Args& a, int32_t n_pages, cudaStream_t st) {
    const size_t slice = bitmap_bytes(n_pages) / kCl;
    const size_t sm = slice <= (size_t)kSliceWords * 4 ? 2 * slice : 0;
    cudaError_t e = cudaSuccess;
    if (sm > 32 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    return e != cudaSuccess ? e : launch_pdl(kern, dim3(kCl), dim3(kPlanThreads), sm, st, a);
}

bool make_caches(Caches* out, const idx_page_cache* caches, int n, int page_size) {
    *out = {};
    out->n = n;
    out->page_size = page_size;
    for (int i = 0; i < n; ++i) {
        const idx_page_cache& c = caches[i];
        out->c[i] = c;
        const uint64_t all = reinterpret_cast<uintptr_t>(c.data) | (uint64_t)c.row_stride_bytes | (uint64_t)c.row_bytes;
        out->vec[i] = all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
        if (c.row_bytes > (INT32_MAX - kSegBytes) / page_size) return false;
        const int64_t segs = ((int64_t)page_size * c.row_bytes + kSegBytes - 1) / kSegBytes;
        out->segs[i] = (int32_t)segs;
        out->segs_total += (int32_t)segs;
    }
    return true;
}

cudaError_t copy_pages(const Caches& cs, const Moves& m, int64_t most, int32_t n_pages, cudaStream_t st) {
    if (cs.segs_total == 0 || most == 0) return cudaSuccess;
    const int64_t work = most > INT64_MAX / cs.segs_total ? INT64_MAX : most * cs.segs_total;
    // many short CTAs: 4096 pages of 90112 bytes take 111 us (6.65 TB/s, 98 % of a plain copy) as 400 per SM, 116 as
    // 16, 122 with 256 threads and 8
    const int64_t grid = (int64_t)sm_count() * 400;
    return launch_pdl(page_copy_kernel, dim3((unsigned)(work < grid ? work : grid)), dim3(kCopyThreads), 0, st, cs, m,
                      n_pages, device_status_ptr());
}

}  // namespace

size_t page_workspace_bytes(int64_t n_seq, int64_t n_pages) {
    // bitmap (whole slices), then the update's free list and per-row arrays, or the compaction's moves and numbers
    const size_t update = align16((size_t)n_pages * 4) + 4 * align16((size_t)n_seq * 4);
    const size_t compact = bitmap_bytes(n_pages) + align16((size_t)n_pages * 4) + 2 * align16(((size_t)n_pages / 2 + 1) * 4) + 16;
    return bitmap_bytes(n_pages) + (update > compact ? update : compact);
}

bool page_caches_fit(const idx_page_cache* caches, int n, int page_size) {
    Caches cs;
    return make_caches(&cs, caches, n, page_size);
}

cudaError_t launch_page_copy(const idx_page_cache* caches, int n_caches, int page_size, int32_t n_pages,
                             const int32_t* src, const int32_t* dst, int32_t n, cudaStream_t st) {
    Caches cs;
    if (!make_caches(&cs, caches, n_caches, page_size)) return cudaErrorNotSupported;
    Moves m = {src, dst, nullptr, nullptr, n};
    return copy_pages(cs, m, n, n_pages, st);
}

cudaError_t launch_page_update(const int32_t* table, int64_t stride, int32_t cols, int32_t n_old, const int32_t* parent,
                               const int32_t* keep, const int32_t* len, int32_t n_seq, int32_t ps, int32_t n_pages,
                               const uint8_t* held, int32_t* out, int64_t out_stride, int32_t out_cols,
                               int32_t* n_free, const idx_page_cache* caches, int n_caches, void* ws, cudaStream_t st) {
    Caches cs;
    if (!make_caches(&cs, caches, n_caches, ps)) return cudaErrorNotSupported;
    uint8_t* w = static_cast<uint8_t*>(ws);
    auto take = [&](size_t bytes) {
        void* p = w;
        w += align16(bytes);
        return p;
    };
    UpdateArgs a = {table, stride, cols, n_old, parent, keep, len, n_seq, ps, n_pages, held, out, out_stride, out_cols,
                    n_free};
    a.bm = static_cast<uint32_t*>(take(bitmap_bytes(n_pages)));
    a.list = static_cast<int32_t*>(take((size_t)n_pages * 4));
    a.offset = static_cast<int32_t*>(take((size_t)n_seq * 4));
    a.src = static_cast<int32_t*>(take((size_t)n_seq * 4));
    a.dst = static_cast<int32_t*>(take((size_t)n_seq * 4));
    a.rows = static_cast<int32_t*>(take((size_t)n_seq * 4));
    a.status = device_status_ptr();
    const cudaError_t e = launch_plan(page_update_kernel, a, n_pages, st);
    if (e != cudaSuccess) return e;
    Moves m = {a.src, a.dst, a.rows, nullptr, n_seq};
    return copy_pages(cs, m, n_seq, n_pages, st);
}

cudaError_t launch_page_compact(const int32_t* table, int64_t stride, int32_t cols, int32_t n_seq, const int32_t* len,
                                int32_t ps, int32_t n_pages, const uint8_t* held, int32_t* out, int64_t out_stride,
                                int32_t* n_used, int32_t* remap, const idx_page_cache* caches, int n_caches, void* ws,
                                cudaStream_t st) {
    Caches cs;
    if (!make_caches(&cs, caches, n_caches, ps)) return cudaErrorNotSupported;
    uint8_t* w = static_cast<uint8_t*>(ws);
    auto take = [&](size_t bytes) {
        void* p = w;
        w += align16(bytes);
        return p;
    };
    CompactArgs a = {table, stride, cols, n_seq, len, ps, n_pages, held, out, out_stride, n_used, remap};
    a.bm = static_cast<uint32_t*>(take(bitmap_bytes(n_pages)));
    a.moving = static_cast<uint32_t*>(take(bitmap_bytes(n_pages)));
    int32_t* numbers = static_cast<int32_t*>(take((size_t)n_pages * 4));
    if (!remap) a.remap = numbers;
    a.src = static_cast<int32_t*>(take(((size_t)n_pages / 2 + 1) * 4));
    a.dst = static_cast<int32_t*>(take(((size_t)n_pages / 2 + 1) * 4));
    a.n_moves = static_cast<int32_t*>(take(4));
    a.status = device_status_ptr();
    const cudaError_t e = launch_plan(page_compact_kernel, a, n_pages, st);
    if (e != cudaSuccess) return e;
    Moves m = {a.src, a.dst, nullptr, a.n_moves, 0};
    return copy_pages(cs, m, n_pages / 2, n_pages, st);
}

}  // namespace lidx
