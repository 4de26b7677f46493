// The pages of paged caches: copying listed pages, a step's update of a page
// table (free, truncate, fork, grow) and compaction.
//
// A page is owned by the table rows that name it, so the plan of an update or a
// compaction starts from a bitmap of the named pages; ranks in the bitmap (a
// prefix sum of its words' zero counts) give the k-th free page, so the result
// depends on nothing but the inputs.  The plan runs on one CTA; the page
// contents then move in a second launch over all SMs.
#include "lidx_internal.cuh"

namespace lidx {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
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
                                           int64_t o0, int64_t o1) {
    constexpr int kBatch = 4;
    constexpr int S = (int)sizeof(V);
    const bool flat = row_bytes == stride;
    for (int64_t o = o0 + (int64_t)threadIdx.x * S; o < o1; o += (int64_t)kCopyThreads * S * kBatch) {
        V v[kBatch];
        int64_t at[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t p = o + (int64_t)i * kCopyThreads * S;
            at[i] = flat ? p : (p / row_bytes) * stride + p % row_bytes;
            if (p < o1) v[i] = *reinterpret_cast<const V*>(src + at[i]);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (o + (int64_t)i * kCopyThreads * S < o1) *reinterpret_cast<V*>(dst + at[i]) = v[i];
    }
}

// a stream of reads and writes: HBM is what bounds it
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(Caches cs, Moves m, int32_t n_pages, int* status) {
    pdl_trigger();
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
        const int64_t end = (int64_t)(m.rows ? m.rows[item] : cs.page_size) * rb;
        const int64_t o0 = (int64_t)seg * kSegBytes;
        const int64_t o1 = o0 + kSegBytes < end ? o0 + kSegBytes : end;
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

// ---------------------------------------------------------------- the plan's pieces (one CTA)

// the exclusive prefix sum of x over the CTA's threads; *total gets the sum
__device__ __forceinline__ int block_scan(int x, int* total) {
    __shared__ int part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();   // part of the last call has been read
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int v = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        part[lane] = v;
    }
    __syncthreads();
    *total = part[31];
    return inc - x + (warp ? part[warp - 1] : 0);
}

// bits of word w that are pages (the last word may be short)
__device__ __forceinline__ uint32_t page_bits(int w, int32_t n_pages) {
    const int64_t left = (int64_t)n_pages - (int64_t)w * 32;
    return left >= 32 ? 0xffffffffu : (1u << left) - 1u;
}

__device__ __forceinline__ uint32_t held_bits(const uint8_t* held, int w, int32_t n_pages) {
    if (!held) return 0u;
    uint32_t x = 0u;
    const int64_t p0 = (int64_t)w * 32;
    for (int i = 0; i < 32 && p0 + i < n_pages; ++i) x |= (held[p0 + i] ? 1u : 0u) << i;
    return x;
}

__device__ __forceinline__ bool bit(const uint32_t* bm, int32_t p) { return (bm[p >> 5] >> (p & 31)) & 1u; }

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
    int32_t* list;         // [n_pages] free pages in order
    int32_t* offset;       // [n_seq] first new page of the row in the list
    int32_t *src, *dst, *rows;   // [n_seq] the copies (-1: none)
    int* status;
};

__global__ void __launch_bounds__(kPlanThreads) page_update_kernel(UpdateArgs a) {
    const int words = (int)(((int64_t)a.n_pages + 31) / 32);
    const int tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    // nothing moves unless the plan says so
    for (int b = tid; b < a.n_seq; b += kPlanThreads) a.src[b] = a.dst[b] = -1;
    // ---- the requests
    bool bad = false;
    for (int b = tid; b < a.n_seq; b += kPlanThreads) {
        const int32_t p = a.parent[b], k = a.keep[b], n = a.len[b];
        bad |= p < -1 || p >= a.n_old || k < 0 || n < k || (p < 0 && k > 0) ||
               (int64_t)k > (int64_t)a.cols * a.ps || (int64_t)n > (int64_t)a.out_cols * a.ps;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            *a.n_free = INT32_MIN;
            flag(a.status, IDX_ERR_DEVICE_BOUNDS);
        }
        return;
    }
    // ---- pages kept whole (and the held ones)
    for (int w = tid; w < words; w += kPlanThreads) a.bm[w] = held_bits(a.held, w, a.n_pages);
    __syncthreads();
    const int warp = tid >> 5, lane = tid & 31;
    for (int b = warp; b < a.n_seq; b += kPlanThreads / 32) {
        const int whole = a.keep[b] / a.ps, part = a.keep[b] % a.ps;
        const int n = whole + (part ? 1 : 0);
        const int32_t* row = a.table + (int64_t)(n ? a.parent[b] : 0) * a.stride;
        for (int i = lane; i < n; i += 32) {
            const int32_t p = row[i];
            if (p < 0 || p >= a.n_pages)
                bad = true;
            else if (i < whole)
                atomicOr(a.bm + (p >> 5), 1u << (p & 31));
            else
                a.src[b] = p;
        }
    }
    if (__syncthreads_or(bad)) {
        for (int b = tid; b < a.n_seq; b += kPlanThreads) a.src[b] = -1;
        if (tid == 0) {
            *a.n_free = INT32_MIN;
            flag(a.status, IDX_ERR_DEVICE_BOUNDS);
        }
        return;
    }
    // ---- the pages kept in part: the first row that wants one has it, unless it is kept whole or held
    for (int b = tid; b < a.n_seq; b += kPlanThreads) {
        const int32_t p = a.src[b];
        bool stays = p >= 0 && !bit(a.bm, p);
        for (int o = 0; stays && o < b; ++o) stays = a.src[o] != p;
        a.rows[b] = p < 0 || stays ? 0 : a.keep[b] % a.ps;   // rows to copy
    }
    __syncthreads();
    for (int b = tid; b < a.n_seq; b += kPlanThreads) {
        const int32_t p = a.src[b];
        if (p >= 0 && a.rows[b] == 0) atomicOr(a.bm + (p >> 5), 1u << (p & 31));
    }
    // ---- new pages of each row, in order
    int need = 0;
    for (int b0 = 0; b0 < a.n_seq; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int x = 0;
        if (b < a.n_seq) {
            const int pages = (int)(((int64_t)a.len[b] + a.ps - 1) / a.ps);
            x = pages - a.keep[b] / a.ps - (a.src[b] >= 0 && a.rows[b] == 0 ? 1 : 0);
        }
        int total;
        const int at = block_scan(x, &total);
        if (b < a.n_seq) a.offset[b] = need + at;
        need += total;
    }
    // ---- the free pages, in order, as many as are needed
    __syncthreads();
    int n_free = 0;
    for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
        const int w = w0 + tid;
        uint32_t z = w < words ? ~a.bm[w] & page_bits(w, a.n_pages) : 0u;
        int total;
        int at = n_free + block_scan(__popc(z), &total);
        for (; z && at < need; z &= z - 1, ++at) a.list[at] = w * 32 + __ffs((int)z) - 1;
        n_free += total;
    }
    if (tid == 0) *a.n_free = n_free - need;
    if (n_free < need) {
        for (int b = tid; b < a.n_seq; b += kPlanThreads) a.src[b] = -1;
        return;
    }
    __syncthreads();
    // ---- the new rows
    for (int b = warp; b < a.n_seq; b += kPlanThreads / 32) {
        const int whole = a.keep[b] / a.ps;
        const int pages = (int)(((int64_t)a.len[b] + a.ps - 1) / a.ps);
        const bool stays = a.src[b] >= 0 && a.rows[b] == 0;
        const int kept = whole + (stays ? 1 : 0);
        const int32_t* row = a.table + (int64_t)(kept ? a.parent[b] : 0) * a.stride;
        const int32_t* list = a.list + a.offset[b] - kept;
        int32_t* out = a.out + (int64_t)b * a.out_stride;
        for (int i = lane; i < a.out_cols; i += 32) out[i] = i < kept ? row[i] : i < pages ? list[i] : -1;
        __syncwarp();
        if (lane == 0) {
            if (stays)
                a.src[b] = -1;
            else if (a.src[b] >= 0)
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
    uint32_t* bm;       // [words] used or held
    int32_t* rank;      // [words] moving pages before the word
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

__global__ void __launch_bounds__(kPlanThreads) page_compact_kernel(CompactArgs a) {
    const int words = (int)(((int64_t)a.n_pages + 31) / 32);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_trigger();
    pdl_wait();
    for (int w = tid; w < words; w += kPlanThreads) a.bm[w] = held_bits(a.held, w, a.n_pages);
    __syncthreads();
    for (int b = warp; b < a.n_seq; b += kPlanThreads / 32) {
        const int n = live_pages(a, b);
        for (int i = lane; i < n; i += 32) {
            const int32_t p = a.table[(int64_t)b * a.stride + i];
            if (p >= 0 && p < a.n_pages)
                atomicOr(a.bm + (p >> 5), 1u << (p & 31));
            else
                flag(a.status, IDX_ERR_DEVICE_BOUNDS);
        }
    }
    __syncthreads();
    int n_used = 0;
    for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
        int total;
        block_scan(w0 + tid < words ? __popc(a.bm[w0 + tid]) : 0, &total);
        n_used += total;
    }
    // the moving pages (used, not held, numbered n_used or higher) and the free numbers below, in order
    int n_moves = 0, n_holes = 0;
    for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
        const int w = w0 + tid;
        uint32_t mv = 0u, ho = 0u;
        if (w < words) {
            const int64_t below = (int64_t)n_used - (int64_t)w * 32;
            const uint32_t low = below >= 32 ? 0xffffffffu : below <= 0 ? 0u : (1u << below) - 1u;
            mv = a.bm[w] & ~held_bits(a.held, w, a.n_pages) & ~low;
            ho = ~a.bm[w] & low;
        }
        int total;
        int at = n_moves + block_scan(__popc(mv), &total);
        if (w < words) a.rank[w] = at;
        for (; mv; mv &= mv - 1, ++at) a.src[at] = w * 32 + __ffs((int)mv) - 1;
        n_moves += total;
        at = n_holes + block_scan(__popc(ho), &total);
        for (; ho; ho &= ho - 1, ++at) a.dst[at] = w * 32 + __ffs((int)ho) - 1;
        n_holes += total;
    }
    if (tid == 0) {
        *a.n_used = n_used;
        *a.n_moves = n_moves;
    }
    __syncthreads();
    // rank of a moving page: those before its word, and those before it in the word
    auto renumber = [&](int32_t p) -> int32_t {
        if (p < n_used || !bit(a.bm, p) || (a.held && a.held[p])) return p;
        const int w = p >> 5;
        const int64_t below = (int64_t)n_used - (int64_t)w * 32;
        const uint32_t low = below <= 0 ? 0u : (1u << below) - 1u;
        const uint32_t mv = a.bm[w] & ~held_bits(a.held, w, a.n_pages) & ~low;
        return a.dst[a.rank[w] + __popc(mv & ((1u << (p & 31)) - 1u))];
    };
    for (int b = warp; b < a.n_seq; b += kPlanThreads / 32) {
        const int n = live_pages(a, b);
        for (int i = lane; i < a.cols; i += 32) {
            int32_t p = -1;
            if (i < n) {
                p = a.table[(int64_t)b * a.stride + i];
                p = p >= 0 && p < a.n_pages ? renumber(p) : -1;
            }
            a.out[(int64_t)b * a.out_stride + i] = p;
        }
    }
    if (a.remap)
        for (int32_t p = tid; p < a.n_pages; p += kPlanThreads) a.remap[p] = renumber(p);
}

size_t align16(size_t x) { return (x + 15) & ~size_t(15); }

bool make_caches(Caches* out, const idx_page_cache* caches, int n, int page_size) {
    *out = {};
    out->n = n;
    out->page_size = page_size;
    for (int i = 0; i < n; ++i) {
        const idx_page_cache& c = caches[i];
        out->c[i] = c;
        const uint64_t all = reinterpret_cast<uintptr_t>(c.data) | (uint64_t)c.row_stride_bytes | (uint64_t)c.row_bytes;
        out->vec[i] = all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
        const int64_t segs = ((int64_t)page_size * c.row_bytes + kSegBytes - 1) / kSegBytes;
        if (segs + out->segs_total > INT32_MAX) return false;
        out->segs[i] = (int32_t)segs;
        out->segs_total += (int32_t)segs;
    }
    return true;
}

cudaError_t copy_pages(const Caches& cs, const Moves& m, int64_t most, int32_t n_pages, cudaStream_t st) {
    if (cs.segs_total == 0 || most == 0) return cudaSuccess;
    const int64_t work = most > INT64_MAX / cs.segs_total ? INT64_MAX : most * cs.segs_total;
    const int64_t grid = (int64_t)sm_count() * 8;
    return launch_pdl(page_copy_kernel, dim3((unsigned)(work < grid ? work : grid)), dim3(kCopyThreads), 0, st, cs, m,
                      n_pages, device_status_ptr());
}

}  // namespace

size_t page_workspace_bytes(int64_t n_seq, int64_t n_pages) {
    const size_t words = (size_t)(n_pages + 31) / 32;
    // bitmap, then the update's free list and per-row arrays, or the compaction's ranks and moves
    const size_t update = align16((size_t)n_pages * 4) + 4 * align16((size_t)n_seq * 4);
    const size_t compact = align16(words * 4) + 2 * align16(((size_t)n_pages / 2 + 1) * 4) + 16;
    return align16(words * 4) + (update > compact ? update : compact);
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
    a.bm = static_cast<uint32_t*>(take(((size_t)n_pages + 31) / 32 * 4));
    a.list = static_cast<int32_t*>(take((size_t)n_pages * 4));
    a.offset = static_cast<int32_t*>(take((size_t)n_seq * 4));
    a.src = static_cast<int32_t*>(take((size_t)n_seq * 4));
    a.dst = static_cast<int32_t*>(take((size_t)n_seq * 4));
    a.rows = static_cast<int32_t*>(take((size_t)n_seq * 4));
    a.status = device_status_ptr();
    cudaError_t e = launch_pdl(page_update_kernel, dim3(1), dim3(kPlanThreads), 0, st, a);
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
    const size_t words = ((size_t)n_pages + 31) / 32;
    CompactArgs a = {table, stride, cols, n_seq, len, ps, n_pages, held, out, out_stride, n_used, remap};
    a.bm = static_cast<uint32_t*>(take(words * 4));
    a.rank = static_cast<int32_t*>(take(words * 4));
    a.src = static_cast<int32_t*>(take(((size_t)n_pages / 2 + 1) * 4));
    a.dst = static_cast<int32_t*>(take(((size_t)n_pages / 2 + 1) * 4));
    a.n_moves = static_cast<int32_t*>(take(4));
    a.status = device_status_ptr();
    cudaError_t e = launch_pdl(page_compact_kernel, dim3(1), dim3(kPlanThreads), 0, st, a);
    if (e != cudaSuccess) return e;
    Moves m = {a.src, a.dst, nullptr, a.n_moves, 0};
    return copy_pages(cs, m, n_pages / 2, n_pages, st);
}

}  // namespace lidx
