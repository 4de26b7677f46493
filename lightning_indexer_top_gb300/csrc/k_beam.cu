// One step of a beam search (idx_beam_step in lidx.h): log-softmax, selection over
// beams and vocabulary, reordering of the token histories.
//
// The logits are read once.  A CTA owns a chunk of a row in registers: its maximum,
// the sum of exponentials, and its n_out best tokens.  The worth of a token within a
// row goes with its logit, so the chunk's list needs no normalisation; a second kernel,
// a CTA per sequence, joins the sums and takes the n_out best of all lists, in 64 bits.
//
// The best K of N keys, K <= 32: a bound that at least K keys reach is cheap - the
// least over W warps of the (K/W)-th best of the lanes' maxima, or the K-th best lane of
// one warp, whichever is higher; each is a sort of 32 lanes in registers.  The few keys
// that reach it go to a list in shared memory and are ranked by counting.  Keys hold
// the column below the logit, so that they differ and ties go to the lower token.  Where
// too many reach the bound (a row of equal logits) K rounds of a maximum are taken instead.
#include "beam.cuh"
#include "sm100_ptx.cuh"

namespace lidx {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;             // scan
constexpr int kMergeThreads = 512, kMergeWarps = kMergeThreads / 32;
constexpr int kList = 1024, kMergeList = 2048;
constexpr float kLog2e = 1.4426950408889634f;

struct Part {
    float m, s;      // maximum (+inf: the row has no worths), sum of exp(x - m)
};

struct BeamArgs {
    idx_beam b;
    int32_t seqs, beams, out, vocab, end, chunks;
    Part* parts;               // [row][chunk]
    unsigned long long* cand;  // [row][chunk][out]: order_key << 32 | ~column, best first; 0: none
    int* status;
};

__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// The bound from the lanes' best keys of all W warps (0: an empty lane); tops[2 * W] in shared memory
template <int W, typename K>
__device__ __forceinline__ K reached_by(K best, int k, K* tops) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // bitonic sort, largest in lane 0
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d; d >>= 1) {
            const K other = __shfl_xor_sync(0xffffffffu, best, d);
            const bool keep_large = ((lane & d) == 0) == ((lane & size) == 0);
            best = keep_large == (best > other) ? best : other;
        }
    if (lane == (k + W - 1) / W - 1) tops[warp] = best;
    if (lane == k - 1) tops[W + warp] = best;
    __syncthreads();
    K least = tops[0], high = tops[W];
#pragma unroll
    for (int i = 1; i < W; ++i) {
        least = min(least, tops[i]);
        high = max(high, tops[W + i]);
    }
    return max(least, high);
}

// E logits a thread; V of them to a load
template <typename T, int E, int V>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(BeamArgs a) {
    __shared__ uint32_t tops[2 * kWarps];
    __shared__ float red[kWarps];
    __shared__ float sums[kWarps];
    __shared__ unsigned long long list[kList];
    __shared__ unsigned long long best_s[kWarps];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t at = blockIdx.x, row = at / a.chunks;
    const int c0 = (int)(at - row * a.chunks) * (kThreads * E);
    pdl_trigger();     // (the merge waits for this kernel's end)
    pdl_wait();
    if (a.b.done && a.b.done[row]) return;
    const T* x = static_cast<const T*>(a.b.logits) + row * a.b.logit_stride;
    float v[E];
#pragma unroll
    for (int p = 0; p < E / V; ++p) {
        const int c = c0 + (p * kThreads + tid) * V;
        if constexpr (V > 1) {
            T y[V];
            if (c + V <= a.vocab) {
                *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(x + c);
#pragma unroll
                for (int i = 0; i < V; ++i) v[p * V + i] = to_f32(y[i]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) v[p * V + i] = c + i < a.vocab ? to_f32(x[c + i]) : -INFINITY;
            }
        } else {
            v[p] = c < a.vocab ? to_f32(x[c]) : -INFINITY;
        }
    }
    auto column = [&](int e) { return c0 + (e / V * kThreads + tid) * V + e % V; };
    float m = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        bad |= !(v[e] < INFINITY);
        m = fmaxf(m, v[e]);
    }
    const uint32_t mine = m > -INFINITY ? order_key(m) : 0u;
    const uint32_t wbest = __reduce_max_sync(0xffffffffu, mine);
    if (lane == 0) red[warp] = wbest ? key_value(wbest) : -INFINITY;
    if (tid == 0) count = 0;
    bad = __syncthreads_or(bad);
    if (bad) {
        if (tid == 0) a.parts[at] = {INFINITY, 0.f};
        return;
    }
    float M = red[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) M = fmaxf(M, red[i]);
    if (M == -INFINITY) {
        if (tid == 0) a.parts[at] = {-INFINITY, 0.f};
        for (int i = tid; i < a.out; i += kThreads) a.cand[at * a.out + i] = 0ull;
        return;
    }
    // sum of exponentials (four chains; the differences are exact enough: |x - M| * 2^-24 of a weight e^-|x - M|)
    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) s4[e & 3] += sm100::ex2_approx((v[e] - M) * kLog2e);
    float s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sums[warp] = s;
    // the best
    const uint32_t bound = max(reached_by<kWarps>(mine, a.out, tops), 1u);
    if (mine >= bound) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t k = v[e] > -INFINITY ? order_key(v[e]) : 0u;
            if (k >= bound) {
                const int i = atomicAdd(&count, 1);
                if (i < kList) list[i] = (unsigned long long)k << 32 | (uint32_t)~column(e);
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) t += sums[i];
        a.parts[at] = {M, t};
    }
    const int n = count;
    unsigned long long* out = a.cand + at * a.out;
    if (n <= kList) {
        for (int i = tid; i < n; i += kThreads) {
            const unsigned long long k = list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += list[j] > k;
            if (rank < a.out) out[rank] = k;
        }
        for (int i = n + tid; i < a.out; i += kThreads) out[i] = 0ull;
        return;
    }
    unsigned long long last = ~0ull;
    for (int r = 0; r < a.out; ++r) {
        unsigned long long best = 0ull;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const unsigned long long k = v[e] > -INFINITY ? (unsigned long long)order_key(v[e]) << 32 | (uint32_t)~column(e) : 0ull;
            if (k < last && k > best) best = k;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        if (lane == 0) best_s[warp] = best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) best = max(best, best_s[i]);
        __syncthreads();
        if (tid == 0) out[r] = best;
        last = best;
    }
}

// order-preserving map of a double (no NaN) to 64 bits, above 0
__device__ __forceinline__ unsigned long long order_key64(double x) {
    const long long u = __double_as_longlong(x == 0.0 ? 0.0 : x);
    return u < 0 ? ~(unsigned long long)u : (unsigned long long)u | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_value64(unsigned long long k) {
    return __longlong_as_double((long long)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

struct Cont {          // a continuation: worth, and beam * vocab + token
    unsigned long long key;
    uint32_t at;
    __device__ __forceinline__ bool better(const Cont& o) const { return key > o.key || (key == o.key && at < o.at); }
};

__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(BeamArgs a) {
    __shared__ double lse[kBeamMax];
    __shared__ unsigned long long keys[kMergeList];
    __shared__ uint32_t ats[kMergeList];
    __shared__ unsigned long long tops[2 * kMergeWarps];
    __shared__ Cont won[kBeamOutMax];
    __shared__ Cont best_s[kMergeWarps];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seq = blockIdx.x;
    const int64_t row0 = (int64_t)seq * a.beams;
    pdl_wait();
    if (tid == 0) count = 0;
    // each beam's log of the sum (NaN: no continuations)
    for (int w = warp; w < a.beams; w += kMergeWarps) {
        const int64_t row = row0 + w;
        const float score = a.b.scores[row];
        const bool done = a.b.done && a.b.done[row];
        bool wrong = !(score < INFINITY);
        float m = -INFINITY;
        const Part* p = a.parts + row * a.chunks;
        if (!done)
            for (int c = lane; c < a.chunks; c += 32) m = fmaxf(m, p[c].m);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double s = 0.0;
        if (!done && m > -INFINITY && m < INFINITY)
            for (int c = lane; c < a.chunks; c += 32)
                if (p[c].m > -INFINITY) s += (double)p[c].s * (double)exp2f((p[c].m - m) * kLog2e);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        wrong |= m == INFINITY;
        if (lane == 0) {
            if (wrong) flag(a.status, IDX_ERR_INEXACT);
            const bool none = wrong || score == -INFINITY || (!done && m == -INFINITY);
            lse[w] = none ? __longlong_as_double(0x7ff8000000000000ll) : done ? 0.0 : (double)m + log(s);
        }
    }
    __syncthreads();
    // lists: one per (beam, chunk), for a beam that is done a single entry
    const int lists = a.beams * a.chunks;
    auto entry = [&](int l, int i) -> Cont {
        const int w = l / a.chunks, c = l - w * a.chunks;
        const double z = lse[w];
        if (z != z) return {0ull, 0u};
        const int64_t row = row0 + w;
        const double base = (double)a.b.scores[row];
        if (a.b.done && a.b.done[row]) {
            if (c || i) return {0ull, 0u};
            return {order_key64(base), (uint32_t)w * (uint32_t)a.vocab + (uint32_t)a.end};
        }
        const unsigned long long k = a.cand[(row * a.chunks + c) * a.out + i];
        if (!k) return {0ull, 0u};
        return {order_key64(base + ((double)key_value((uint32_t)(k >> 32)) - z)),
                (uint32_t)w * (uint32_t)a.vocab + ~(uint32_t)k};
    };
    unsigned long long mine = 0ull;
    for (int l = tid; l < lists; l += kMergeThreads) mine = max(mine, entry(l, 0).key);
    const unsigned long long bound = max(reached_by<kMergeWarps>(mine, a.out, tops), 1ull);
    if (mine >= bound)
        for (int l = tid; l < lists; l += kMergeThreads)
            for (int i = 0; i < a.out; ++i) {
                const Cont e = entry(l, i);
                if (e.key < bound) break;
                const int j = atomicAdd(&count, 1);
                if (j < kMergeList) {
                    keys[j] = e.key;
                    ats[j] = e.at;
                }
            }
    if (tid < a.out) won[tid] = {0ull, 0u};
    __syncthreads();
    const int n = count;
    if (n <= kMergeList) {
        for (int i = tid; i < n; i += kMergeThreads) {
            const Cont e = {keys[i], ats[i]};
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += Cont{keys[j], ats[j]}.better(e);
            if (rank < a.out) won[rank] = e;
        }
        __syncthreads();
    } else {
        Cont last = {~0ull, 0u};
        for (int r = 0; r < a.out; ++r) {
            Cont best = {0ull, 0u};
            for (int l = tid; l < lists; l += kMergeThreads)
                for (int i = 0; i < a.out; ++i) {
                    const Cont e = entry(l, i);
                    if (!e.key) break;
                    if (last.better(e)) {      // (a list's entries come best first: the first one below is its best)
                        if (e.better(best)) best = e;
                        break;
                    }
                }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const Cont e = {__shfl_xor_sync(0xffffffffu, best.key, o), __shfl_xor_sync(0xffffffffu, best.at, o)};
                if (e.better(best)) best = e;
            }
            if (lane == 0) best_s[warp] = best;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kMergeWarps; ++i)
                if (best_s[i].better(best)) best = best_s[i];
            __syncthreads();
            if (tid == 0) won[r] = best;
            if (!best.key) break;
            last = best;
        }
        __syncthreads();
    }
    // results; a warp per kept continuation copies its history
    for (int r = warp; r < a.out; r += kMergeWarps) {
        const Cont e = won[r];
        const int64_t to = (int64_t)seq * a.out + r;
        const bool none = e.key == 0ull;
        const int w = none ? 0 : (int)(e.at / (uint32_t)a.vocab), token = none ? -1 : (int)(e.at - (uint32_t)w * (uint32_t)a.vocab);
        const int64_t row = row0 + w;
        const bool was = !none && a.b.done && a.b.done[row];
        if (lane == 0) {
            a.b.out_scores[to] = none ? -INFINITY : (float)key_value64(e.key);
            a.b.parent[to] = none ? -1 : (int32_t)row;
            a.b.token[to] = token;
            a.b.out_done[to] = none || was || token == a.end;
        }
        if (!a.b.lengths) continue;
        int len = none ? 0 : a.b.lengths[row];
        const int room = a.b.history_cols;
        bool grows = !none && !was;
        if (len < 0 || len > room || (grows && len >= room)) {
            if (lane == 0) flag(a.status, IDX_ERR_DEVICE_BOUNDS);
            grows = false;
            len = min(max(len, 0), room);
        }
        const int32_t* src = a.b.history + row * a.b.history_stride;
        int32_t* dst = a.b.out_history + to * a.b.out_history_stride;
#pragma unroll 4
        for (int i = lane; i < len; i += 32) dst[i] = src[i];
        if (lane == 0) {
            if (grows) dst[len] = token;
            a.b.out_lengths[to] = len + grows;
        }
    }
}

int64_t chunk_of(int64_t rows, int64_t vocab) {
    // short chunks while long ones would leave SMs without work
    return rows * ((vocab + 32 * kThreads - 1) / (32 * kThreads)) < 2 * 152 ? 8 * kThreads : 32 * kThreads;
}

template <typename T, int E>
cudaError_t scan(const BeamArgs& a, bool vec, cudaStream_t st) {
    const int64_t ctas = (int64_t)a.seqs * a.beams * a.chunks;
    if (ctas > INT32_MAX) return cudaErrorNotSupported;
    const dim3 grid((unsigned)ctas);
    return vec ? launch_pdl(beam_scan_kernel<T, E, 16 / (int)sizeof(T)>, grid, dim3(kThreads), 0, st, a)
               : launch_pdl(beam_scan_kernel<T, E, 1>, grid, dim3(kThreads), 0, st, a);
}

template <typename T>
cudaError_t run(const BeamArgs& a, cudaStream_t st) {
    // (one order of a row's elements for every row of the call: equal rows get equal sums)
    const bool vec = reinterpret_cast<uintptr_t>(a.b.logits) % 16 == 0 && a.b.logit_stride * (int64_t)sizeof(T) % 16 == 0;
    cudaError_t e = chunk_of((int64_t)a.seqs * a.beams, a.vocab) == 8 * kThreads ? scan<T, 8>(a, vec, st) : scan<T, 32>(a, vec, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(beam_merge_kernel, dim3((unsigned)a.seqs), dim3(kMergeThreads), 0, st, a);
}

}  // namespace

int64_t beam_workspace_bytes(int64_t seqs, int64_t beams, int64_t out, int64_t vocab) {
    const int64_t rows = seqs * beams, chunk = chunk_of(rows, vocab), chunks = (vocab + chunk - 1) / chunk;
    return rows * chunks * (int64_t)(sizeof(Part) + out * sizeof(unsigned long long));
}

cudaError_t launch_beam(const idx_beam& b, int dtype, int seqs, int beams, int out, int vocab, int end, void* ws, cudaStream_t st) {
    BeamArgs a = {};
    a.b = b;
    a.seqs = seqs;
    a.beams = beams;
    a.out = out;
    a.vocab = vocab;
    a.end = end;
    const int64_t rows = (int64_t)seqs * beams, chunk = chunk_of(rows, vocab);
    a.chunks = (int)((vocab + chunk - 1) / chunk);
    a.parts = static_cast<Part*>(ws);
    a.cand = reinterpret_cast<unsigned long long*>(a.parts + rows * a.chunks);
    a.status = device_status_ptr();
    switch (dtype) {
        case IDX_F16: return run<__half>(a, st);
        case IDX_BF16: return run<__nv_bfloat16>(a, st);
        default: return run<float>(a, st);
    }
}

}  // namespace lidx
