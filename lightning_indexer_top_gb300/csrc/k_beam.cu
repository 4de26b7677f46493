// One step of a beam search (idx_beam_step in lidx.h): log-softmax, selection over
// beams and vocabulary, reordering of the token histories.
//
// The logits are read once.  A CTA owns a chunk of a row in registers: its maximum,
// the sum of exponentials, and its n_out best tokens.  The worth of a token within a
// row goes with its logit, so the chunk's list needs no normalisation; a second kernel,
// a CTA per sequence, joins the sums and takes the n_out best of all lists, in 64 bits.
// Where these round different logits to one worth (a beam's score of -3e38, say), lists may
// have left out tokens that are worth as much as the last one kept: their chunks are then
// looked through for the lowest ones.
//
// The best K of N keys, K <= 32: a bound that at least K keys reach is cheap, the least over W warps of the (K/W)-th best
// of the lanes' maxima.  The few keys that reach it go to a list in shared memory and are ranked by counting.  Keys hold
// the column below the logit, so that they differ and ties go to the lower token.  Where too many reach the bound (a row
// of equal logits) K rounds of a maximum are taken instead.
//
// The scan waits more than it works (seven instructions a logit): 16-bit logits stay packed so that more CTAs are at it,
// sums run against the warp's maximum so that two barriers are enough.
// 512 rows of 131072 bf16 logits, 16 kept of each eight: 64 us (f32: 81).  By itself the scan takes 40, with issue slots used on 45 %
// of the cycles, and the merge 27, with one CTA to a sequence, which waits at barriers and for one load after another.
#include <float.h>

#include "beam.cuh"
#include "dense_attn.cuh"

namespace lidx {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;             // scan
constexpr int kMergeThreads = 512, kMergeWarps = kMergeThreads / 32;
constexpr int kList = 1024, kMergeList = 2048;

struct Part {
    float m, s;      // maximum (+inf: the row has no worths), sum of exp(x - m)
};

struct BeamArgs {
    idx_beam b;
    int32_t seqs, beams, out, vocab, end, chunks, per_thread, dtype;
    Part* parts;               // [row][chunk]
    unsigned long long* cand;  // [row][chunk][out]: order_key << 32 | ~column, best first; 0: none
    int* status;
};

__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// The lanes' n-th best key, n <= 32 (0: fewer are above 0); first: the best
template <typename K>
__device__ __forceinline__ K nth_of_lanes(K mine, int n, K& first) {
    const int lane = threadIdx.x & 31;
    K best = 0;
    for (int i = 0; i < n; ++i) {
        if constexpr (sizeof(K) == 4) {
            best = __reduce_max_sync(0xffffffffu, mine);
        } else {
            best = mine;
#pragma unroll
            for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        }
        if (i == 0) first = best;
        if (lane == __ffs(__ballot_sync(0xffffffffu, mine == best)) - 1) mine = 0;
    }
    return best;
}

__device__ __forceinline__ float max_of(const float* v, int n) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < n; ++i) m = fmaxf(m, v[i]);
    return m;
}
__device__ __forceinline__ float max_of(const __half* v, int n) {
    __half2 m = *reinterpret_cast<const __half2*>(v);
#pragma unroll
    for (int i = 2; i < n; i += 2) m = __hmax2(m, *reinterpret_cast<const __half2*>(v + i));
    return __half2float(__hmax(__low2half(m), __high2half(m)));
}
__device__ __forceinline__ float max_of(const __nv_bfloat16* v, int n) {
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(v);
#pragma unroll
    for (int i = 2; i < n; i += 2) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(v + i));
    return __bfloat162float(__hmax(__low2bfloat16(m), __high2bfloat16(m)));
}

// Bits of those of the 32 (or fewer) elements from v on that reach r (a number): element e at bit e; of 16-bit ones
// e / 2 + 16 (e % 2)
template <int N>
__device__ __forceinline__ uint32_t reaching(const float* v, float r) {
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < N; ++e) m |= v[e] >= r ? 1u << e : 0u;
    return m;
}
template <int N>
__device__ __forceinline__ uint32_t reaching(const __half* v, float r) {
    const __half2 r2 = __float2half2_rn(fmaxf(r, -65504.f));
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < N; e += 2) m |= __hge2_mask(*reinterpret_cast<const __half2*>(v + e), r2) & (0x10001u << (e / 2));
    return m;
}
template <int N>
__device__ __forceinline__ uint32_t reaching(const __nv_bfloat16* v, float r) {
    const __nv_bfloat162 r2 = __float2bfloat162_rn(fmaxf(r, __uint_as_float(0xff7f0000u)));      // (the lowest finite one)
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < N; e += 2) m |= __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(v + e), r2) & (0x10001u << (e / 2));
    return m;
}

// two numbers as a packed pair of f32
__device__ __forceinline__ uint64_t two(const float* v) { return (uint64_t)__float_as_uint(v[1]) << 32 | __float_as_uint(v[0]); }
__device__ __forceinline__ uint64_t two(const __half* v) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(v));
    return (uint64_t)__float_as_uint(x.y) << 32 | __float_as_uint(x.x);
}
__device__ __forceinline__ uint64_t two(const __nv_bfloat16* v) {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(v);
    return (uint64_t)(x & 0xffff0000u) << 32 | (x << 16);
}

// E logits a thread; V of them to a load
template <typename T, int E, int V>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && E < 64 ? 4 : 3) beam_scan_kernel(BeamArgs a) {
    __shared__ uint32_t tops[kWarps];
    __shared__ float maxima[kWarps], sums[kWarps];
    __shared__ unsigned long long list[kList];
    __shared__ unsigned long long best_s[kWarps];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t at = blockIdx.x, row = blockIdx.x / (unsigned)a.chunks;
    const int c0 = (int)(at - row * a.chunks) * (kThreads * E);
    pdl_trigger();     // (the merge waits for this kernel's end)
    pdl_wait();
    if (a.b.done && a.b.done[row]) return;
    const T* x = static_cast<const T*>(a.b.logits) + row * a.b.logit_stride;
    __align__(16) T v[E];
#pragma unroll
    for (int p = 0; p < E / V; ++p) {
        const int c = c0 + (p * kThreads + tid) * V;
        if (V > 1 && c + V <= a.vocab) {
            *reinterpret_cast<uint4*>(v + p * V) = *reinterpret_cast<const uint4*>(x + c);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[p * V + i] = c + i < a.vocab ? x[c + i] : from_f32<T>(-INFINITY);
        }
    }
    const float m = max_of(v, E);       // (of the numbers; a NaN shows in the sum)
    const uint32_t mine = m > -INFINITY ? order_key(m) : 0u;
    uint32_t first = 0u;
    // (a row's last chunk may leave warps without columns: the others' bound)
    const int full = max(min(kThreads, (a.vocab - c0 + V - 1) / V) / 32, 1);
    const uint32_t nth = nth_of_lanes(mine, (a.out + full - 1) / full, first);
    const float wm = first ? key_value(first) : -INFINITY;
    // sum of exponentials against the warp's maximum (four chains; |x - wm| * 2^-24 of a weight e^-|x - wm|)
    const float ref = first ? wm : 0.f;
    const uint64_t ref2 = pair(-ref, -ref), log2e2 = pair(kLog2e, kLog2e);
    uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        float x0, x1;
        unpair(mul2(add2(two(v + e), ref2), log2e2), x0, x1);
        s2[e / 2 & 1] = add2(s2[e / 2 & 1], pair(sm100::ex2_approx(x0), sm100::ex2_approx(x1)));
    }
    float s, s_odd;
    unpair(add2(s2[0], s2[1]), s, s_odd);
    s += s_odd;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
        maxima[warp] = wm;
        sums[warp] = s;
        tops[warp] = nth;
    }
    if (tid == 0) count = 0;
    __syncthreads();
    float M = maxima[0];
    uint32_t bound = tops[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
        M = fmaxf(M, maxima[i]);
        if (i < full) bound = min(bound, tops[i]);
    }
    // (as a number, at least the lowest finite one: neither -inf nor a NaN reaches it)
    const float reach = key_value(max(bound, order_key(-FLT_MAX)));
    if (m >= reach) {
        constexpr int kGroup = E < 32 ? E : 32;
#pragma unroll
        for (int g = 0; g < E; g += kGroup)
            for (uint32_t left = reaching<kGroup>(v + g, reach); left; left &= left - 1) {
                const int bit = __ffs(left) - 1, e = g + (sizeof(T) == 2 ? 2 * (bit & 15) + (bit >> 4) : bit);
                const int c = c0 + (e / V * kThreads + tid) * V + e % V;
                const int i = atomicAdd(&count, 1);
                if (i < kList) list[i] = (unsigned long long)order_key(to_f32(x[c])) << 32 | (uint32_t)~c;      // (read again: few are)
            }
    }
    __syncthreads();
    if (tid == 0) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
            t += sums[i] * (maxima[i] > -INFINITY ? sm100::ex2_approx((maxima[i] - M) * kLog2e) : sums[i] != sums[i] ? 1.f : 0.f);
        a.parts[at] = {M < INFINITY && t == t ? M : INFINITY, t};
    }
    const int n = count;
    unsigned long long* out = a.cand + at * a.out;
    if (n <= kList) {
        for (int i = tid; i < n; i += kThreads) {
            const unsigned long long k = list[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) rank += list[j] > k;
            if (rank < a.out) out[rank] = k;
        }
        for (int i = n + tid; i < a.out; i += kThreads) out[i] = 0ull;
        return;
    }
    // (the logits are read again: kept until here they would cost every CTA registers)
    unsigned long long last = ~0ull;
    for (int r = 0; r < a.out; ++r) {
        unsigned long long best = 0ull;
        for (int i = tid; i < kThreads * E && c0 + i < a.vocab; i += kThreads) {
            const float y = to_f32(x[c0 + i]);
            const unsigned long long k = y > -INFINITY ? (unsigned long long)order_key(y) << 32 | (uint32_t)~(c0 + i) : 0ull;
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
    __shared__ double lse[kBeamMax];       // of a beam's logits; 0 of one that is done; NaN: no continuations
    __shared__ float base[kBeamMax];       // its score
    __shared__ uint8_t ended[kBeamMax];    // whether it is done
    __shared__ float top[kBeamMax];        // its largest logit
    __shared__ int lens[kBeamMax];         // its history's length
    __shared__ unsigned long long keys[kMergeList];
    __shared__ uint32_t ats[kMergeList];
    __shared__ unsigned long long tops[kMergeWarps];
    __shared__ Cont won[kBeamOutMax];
    __shared__ Cont best_s[kMergeWarps];
    __shared__ int count;
    __shared__ unsigned long long hidden;      // the largest worth that full lists may have left out
    __shared__ uint32_t marks[kMergeWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seq = blockIdx.x;
    const int64_t row0 = (int64_t)seq * a.beams;
    pdl_wait();
    if (tid == 0) {
        count = 0;
        hidden = 0ull;
    }
    const int lists = a.beams * a.chunks;
    // lists are dealt to as many warps as they fill, one after the other, so that the warps have about as many.  (To all warps, with
    // fewer lists each: a bound so low that 110 us were taken for 64.)
    const int warps = min((lists + 31) / 32, kMergeWarps);
    const int mine_at = warp + warps * lane;
    const bool has = warp < warps && mine_at < lists;
    const unsigned long long head = has ? a.cand[(row0 * a.chunks + mine_at) * a.out] : 0ull;      // (on its way meanwhile)
    for (int w = warp; w < a.beams; w += kMergeWarps) {
        const int64_t row = row0 + w;
        const float score = a.b.scores[row];
        const bool done = a.b.done && a.b.done[row];
        float m = -INFINITY;
        const Part* p = a.parts + row * a.chunks;
        // (what a beam that is done has there is not looked at, but not waited for either)
        Part first = lane < a.chunks ? p[lane] : Part{-INFINITY, 0.f};
        const int len = a.b.lengths ? a.b.lengths[row] : 0;
        if (done) first.m = -INFINITY;
        m = first.m;
        if (!done)
            for (int c = lane + 32; c < a.chunks; c += 32) m = fmaxf(m, p[c].m);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double s = 0.0;
        if (m > -INFINITY && m < INFINITY) {
            if (first.m > -INFINITY) s = (double)(first.s * exp2f((first.m - m) * kLog2e));
            for (int c = lane + 32; c < a.chunks; c += 32)
                if (p[c].m > -INFINITY) s += (double)(p[c].s * exp2f((p[c].m - m) * kLog2e));
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        }
        if (lane == 0) {
            base[w] = score;
            ended[w] = done;
            lens[w] = len;
            top[w] = m;
            lse[w] = s;
        }
    }
    __syncthreads();
    // (64-bit logarithms are slow here: a lane to a beam)
    for (int w = tid; w < a.beams; w += kMergeThreads) {
        const float score = base[w], m = top[w];
        const bool wrong = !(score < INFINITY) || m == INFINITY, none = wrong || score == -INFINITY || (!ended[w] && m == -INFINITY);
        if (wrong) flag(a.status, IDX_ERR_INEXACT);
        lse[w] = none ? __longlong_as_double(0x7ff8000000000000ll) : ended[w] ? 0.0 : (double)m + log(lse[w]);
    }
    __syncthreads();
    // lists: one per (beam, chunk), for a beam that is done a single entry
    auto value = [&](int l, int i, unsigned long long k) -> Cont {       // k: what the list has there
        const int w = l / a.chunks, c = l - w * a.chunks;
        const double z = lse[w];
        if (z != z) return {0ull, 0u};
        if (ended[w]) {
            if (c || i) return {0ull, 0u};
            return {order_key64((double)base[w]), (uint32_t)w * (uint32_t)a.vocab + (uint32_t)a.end};
        }
        if (!k) return {0ull, 0u};
        return {order_key64((double)base[w] + ((double)key_value((uint32_t)(k >> 32)) - z)),
                (uint32_t)w * (uint32_t)a.vocab + ~(uint32_t)k};
    };
    const unsigned long long* cand = a.cand + row0 * a.chunks * a.out;
    auto entry = [&](int l, int i) -> Cont { return value(l, i, cand[(int64_t)l * a.out + i]); };
    unsigned long long mine = has ? value(mine_at, 0, head).key : 0ull, first = 0ull;
    if (warp < warps)
        for (int l = mine_at + warps * 32; l < lists; l += warps * 32) mine = max(mine, entry(l, 0).key);
    const unsigned long long nth = nth_of_lanes(mine, (a.out + warps - 1) / warps, first);
    if (lane == 0) tops[warp] = nth;
    __syncthreads();
    unsigned long long bound = tops[0];
    for (int i = 1; i < warps; ++i) bound = min(bound, tops[i]);
    bound = max(bound, 1ull);
    if (mine >= bound && warp < warps)
        for (int l = mine_at; l < lists; l += warps * 32) {
            bool on = true;
            for (int i0 = 0; on && i0 < a.out; i0 += 4) {
                unsigned long long k[4];      // four at a time
#pragma unroll
                for (int i = 0; i < 4; ++i) k[i] = i0 + i < a.out ? cand[(int64_t)l * a.out + i0 + i] : 0ull;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!on || i0 + i >= a.out) break;
                    const Cont e = value(l, i0 + i, k[i]);
                    on = e.key >= bound;
                    if (!on) break;
                    const int j = atomicAdd(&count, 1);
                    if (j < kMergeList) {
                        keys[j] = e.key;
                        ats[j] = e.at;
                    }
                    // (a list's last entry: whether the next logit below it would be worth as much)
                    if (i0 + i == a.out - 1 && !ended[l / a.chunks] && value(l, 0, k[i] - (1ull << 32)).key == e.key)
                        atomicMax(&hidden, e.key);
                }
            }
        }
    if (tid < a.out) won[tid] = {0ull, 0u};
    __syncthreads();
    const int n = count;
    if (n <= kMergeList) {
        for (int i = tid; i < n; i += kMergeThreads) {
            const Cont e = {keys[i], ats[i]};
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) rank += Cont{keys[j], ats[j]}.better(e);
            if (rank < a.out) won[rank] = e;
        }
        __syncthreads();
    } else {
        // (by worth and place in the lists, which is the order that every list has)
        Cont last = {~0ull, 0u};
        for (int r = 0; r < a.out; ++r) {
            Cont best = {0ull, 0u};
            for (int l = tid; l < lists; l += kMergeThreads)
                for (int i = 0; i < a.out; ++i) {
                    const Cont e = {entry(l, i).key, (uint32_t)l * a.out + i};
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
            if (tid == 0) won[r] = {best.key, best.key ? entry(best.at / a.out, best.at % a.out).at : 0u};
            if (!best.key) break;
            last = best;
        }
        __syncthreads();
    }
    const unsigned long long least = won[a.out - 1].key;
    if (least && (n > kMergeList || hidden == least)) {
        // What is worth more than the last one kept is there; of what is worth as much, the lowest beams and tokens, from the
        // logits.  A list whose first entry is worth that gives one at least, the others hold what is worth more: fewer than
        // 2 out chunks are read.
        Cont mine_won = {0ull, 0u};
        int have = 0, rank = 0;
        if (tid < a.out) mine_won = won[tid];
        for (int r = 0; r < a.out; ++r) {
            have += won[r].key > least;
            rank += won[r].better(mine_won);
        }
        __syncthreads();
        if (mine_won.key > least) won[rank] = mine_won;
        const int chunk = a.per_thread * kThreads;
        for (int l0 = 0; l0 < lists && have < a.out; l0 += kMergeThreads) {
            __syncthreads();
            const uint32_t mark = __ballot_sync(0xffffffffu, l0 + tid < lists && entry(l0 + tid, 0).key >= least);
            if (lane == 0) best_s[warp].at = mark;
            __syncthreads();
            for (int i = 0; i < kMergeWarps; ++i)
                for (uint32_t left = best_s[i].at; left && have < a.out; left &= left - 1) {
                    const int l = l0 + 32 * i + __ffs(left) - 1, w = l / a.chunks;
                    const int first = ended[w] ? 0 : (l - w * a.chunks) * chunk, past = ended[w] ? 1 : min(first + chunk, a.vocab);
                    for (int t0 = first; t0 < past && have < a.out; t0 += kMergeThreads) {
                        const int t = t0 + tid;
                        Cont e = {0ull, 0u};
                        if (t < past && ended[w]) {
                            e = value(l, 0, 0ull);
                        } else if (t < past) {
                            const int64_t at = (row0 + w) * a.b.logit_stride + t;
                            const float x = a.dtype == IDX_F32   ? static_cast<const float*>(a.b.logits)[at]
                                            : a.dtype == IDX_F16 ? to_f32(static_cast<const __half*>(a.b.logits)[at])
                                                                 : to_f32(static_cast<const __nv_bfloat16*>(a.b.logits)[at]);
                            e = value(l, 0, x > -INFINITY ? (unsigned long long)order_key(x) << 32 | (uint32_t)~t : 0ull);
                        }
                        const uint32_t hit = __ballot_sync(0xffffffffu, e.key == least);
                        if (lane == 0) marks[warp] = hit;
                        __syncthreads();
                        int at = have;
                        for (int v = 0; v < kMergeWarps; ++v) {
                            if (v < warp) at += __popc(marks[v]);
                            have += __popc(marks[v]);
                        }
                        at += __popc(hit & ((1u << lane) - 1u));
                        if (e.key == least && at < a.out) won[at] = e;
                        __syncthreads();
                    }
                }
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
        const bool was = !none && ended[w];
        if (lane == 0) {
            a.b.out_scores[to] = none ? -INFINITY : (float)key_value64(e.key);
            a.b.parent[to] = none ? -1 : (int32_t)row;
            a.b.token[to] = token;
            a.b.out_done[to] = none || was || token == a.end;
        }
        if (!a.b.lengths) continue;
        int len = none ? 0 : lens[w];
        const int room = a.b.history_cols;
        bool grows = !none && !was;
        if (len < 0 || len > room || (grows && len >= room)) {
            if (lane == 0) flag(a.status, IDX_ERR_DEVICE_BOUNDS);
            grows = false;
            len = min(max(len, 0), room);
        }
        const int32_t* src = a.b.history + row * a.b.history_stride;
        int32_t* dst = a.b.out_history + to * a.b.out_history_stride;
        int from = 0;
        if (((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15u) == 0) {
#pragma unroll 4
            for (int i = lane; i < len / 4; i += 32) reinterpret_cast<int4*>(dst)[i] = reinterpret_cast<const int4*>(src)[i];
            from = len / 4 * 4;
        }
#pragma unroll 4
        for (int i = from + lane; i < len; i += 32) dst[i] = src[i];
        if (lane == 0) {
            if (grows) dst[len] = token;
            a.b.out_lengths[to] = len + grows;
        }
    }
}

// Logits to a thread: few while more would leave SMs without work, many where there is plenty (a CTA's barriers and its list
// take as long whatever it holds).  8, 32 and 64 of them: 4 f32 rows of 32000 9.3, 10.6 us; 16 of them 13.5, 23.7; 32 bf16 rows of
// 32000 11.3, 15.1, 16.0; 64 bf16 rows of 131072 28.9, 16.2, 16.6; 512 of them 128, 66.6, 63.5 (f32: 131, 81.9).  Not the best
// for few long rows: 8 bf16 rows of 131072 15.5, 11.0, 12.7.
int logits_of(int64_t rows, int64_t vocab, int dtype) {
    auto ctas = [&](int n) { return rows * ((vocab + n * kThreads - 1) / (n * kThreads)); };
    return ctas(32) < 2 * 152 ? 8 : dtype != IDX_F32 && ctas(64) >= 8 * 152 ? 64 : 32;
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
    cudaError_t e;
    switch (a.per_thread) {
        case 8: e = scan<T, 8>(a, vec, st); break;
        case 32: e = scan<T, 32>(a, vec, st); break;
        default: e = scan<T, sizeof(T) == 2 ? 64 : 32>(a, vec, st);
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(beam_merge_kernel, dim3((unsigned)a.seqs), dim3(kMergeThreads), 0, st, a);
}

}  // namespace

int64_t beam_workspace_bytes(int64_t seqs, int64_t beams, int64_t out, int64_t vocab) {
    // (of the type that takes the shorter chunks)
    const int64_t rows = seqs * beams, chunk = logits_of(rows, vocab, IDX_F32) * kThreads, chunks = (vocab + chunk - 1) / chunk;
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
    a.dtype = dtype;
    const int64_t rows = (int64_t)seqs * beams;
    a.per_thread = logits_of(rows, vocab, dtype);
    const int64_t chunk = a.per_thread * kThreads;
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
