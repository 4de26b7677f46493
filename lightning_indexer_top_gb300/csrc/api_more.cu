// C-ABI entry points of the cache writes, of the attention over 4-bit caches and of the beam search's step.
#include <stdarg.h>
#include <stdio.h>

#include <cmath>

#include "beam.cuh"
#include "dense_attn.cuh"
#include "q4.cuh"

namespace lidx {
namespace {

idx_status bad(idx_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return record_error(s, buf);
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool valid_dtype(int t) { return t == IDX_F32 || t == IDX_F16 || t == IDX_BF16; }

// rows of `width` bytes, `pitch` apart, `bytes` from the first to the end of the last
struct Bytes {
    const void* p;
    int64_t bytes, pitch, width;
};

// (rows that lie equally far apart may be columns of one matrix, beside each other)
bool overlap(const Bytes& x, const Bytes& y) {
    if (!x.p || !y.p || !x.bytes || !y.bytes) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    if (a >= b + y.bytes || b >= a + x.bytes) return false;
    if (x.pitch != y.pitch || x.pitch <= 0) return true;
    const int64_t off = a >= b ? (int64_t)((a - b) % x.pitch) : x.pitch - 1 - (int64_t)((b - a - 1) % x.pitch);
    return off < y.width || off + x.width > x.pitch;
}

// a 4-bit cache of n heads of d columns
idx_status check_q4(const char* what, const char* which, const void* cache, int64_t stride, int64_t n, int64_t d) {
    if (stride < q4_payload(n, d))
        return bad(IDX_ERR_INVALID_ARG, "%s: %s rows of %lld bytes need a stride of at least that", what, which,
                   (long long)q4_payload(n, d));
    if (stride % 4 || !aligned(cache, 4))
        return bad(IDX_ERR_INVALID_ARG, "%s: %s and its row stride must be multiples of 4 bytes", what, which);
    return IDX_OK;
}

idx_status append(const char* what, bool q4, const idx_new_rows* rows, idx_dtype dtype, int32_t Hq, int32_t Hkv, int32_t dk,
                  int32_t dv, const idx_batch& batch, const idx_rope* rope, void* k_cache, int64_t kc_stride, void* v_cache,
                  int64_t vc_stride, int64_t kv_rows, cudaStream_t st) {
    idx_status s = validate_batch(batch, what);
    if (s != IDX_OK) return s;
    if (!valid_dtype(dtype)) return bad(IDX_ERR_INVALID_ARG, "%s: bad dtype", what);
    if (!rows) return bad(IDX_ERR_INVALID_ARG, "%s: rows is NULL", what);
    if (Hkv < 1 || Hq < 0) return bad(IDX_ERR_INVALID_ARG, "%s: need n_kv_heads >= 1 and n_q_heads >= 0", what);
    if (dk < 1 || dk > 576 || dv < 0 || dv > 512)
        return bad(IDX_ERR_INVALID_ARG, "%s: need 1 <= dk <= 576 and 0 <= dv <= 512", what);
    const int64_t wide = INT32_MAX / 2;
    if ((int64_t)Hq * dk > wide || (int64_t)Hkv * (dk + dv) > wide) return bad(IDX_ERR_UNSUPPORTED, "%s: rows too wide", what);
    if (q4 && (dk % 8 || dv % 8)) return bad(IDX_ERR_INVALID_ARG, "%s: dk and dv must be multiples of 8", what);
    if (kv_rows < 0) return bad(IDX_ERR_INVALID_ARG, "%s: kv_rows < 0", what);
    AppendArgs a = {};
    if (rope) {
        if (rope->n_rot < 0 || rope->n_rot % 2 || rope->start < 0 || rope->n_rot > dk || rope->start > dk - rope->n_rot)
            return bad(IDX_ERR_INVALID_ARG, "%s: need an even n_rot >= 0 and 0 <= start <= dk - n_rot", what);
        if (rope->n_rot && !rope->inv_freq) return bad(IDX_ERR_INVALID_ARG, "%s: inv_freq is NULL", what);
        a.inv_freq = rope->inv_freq;
        a.n_rot = rope->n_rot;
        a.start = rope->n_rot ? rope->start : 0;
        a.interleaved = rope->n_rot && rope->interleaved;
    }
    a.rows = *rows;
    if (Hq == 0) a.rows.q = nullptr, a.rows.q_out = nullptr, a.rows.q_stride = a.rows.q_out_stride = 0;
    if (dv == 0) {
        if (rows->v || v_cache) return bad(IDX_ERR_INVALID_ARG, "%s: v and v_cache need dv > 0", what);
        a.rows.v_stride = 0;
        vc_stride = 0;
    }
    const int64_t n = (int64_t)batch.n_seq * batch.n_q_per_seq;
    if (a.rows.k_stride < (int64_t)Hkv * dk || (dv && a.rows.v_stride < (int64_t)Hkv * dv) ||
        (Hq && (a.rows.q_stride < (int64_t)Hq * dk || a.rows.q_out_stride < (int64_t)Hq * dk)))
        return bad(IDX_ERR_INVALID_ARG, "%s: a stride of the new rows is below their width", what);
    if (q4) {
        s = check_q4(what, "k_cache", k_cache, kc_stride, Hkv, dk);
        if (s == IDX_OK && dv) s = check_q4(what, "v_cache", v_cache, vc_stride, Hkv, dv);
        if (s != IDX_OK) return s;
    } else if (kc_stride < (int64_t)Hkv * dk || (dv && vc_stride < (int64_t)Hkv * dv)) {
        return bad(IDX_ERR_INVALID_ARG, "%s: a cache's row stride is below its row", what);
    }
    if (n == 0) return IDX_OK;
    if (!rows->k || (dv && !rows->v) || (Hq && (!rows->q || !rows->q_out)))
        return bad(IDX_ERR_INVALID_ARG, "%s: NULL k, v, q or q_out", what);
    if (kv_rows > 0 && (!k_cache || (dv && !v_cache))) return bad(IDX_ERR_INVALID_ARG, "%s: NULL k_cache or v_cache", what);
    if (Hq && a.rows.q == a.rows.q_out && a.rows.q_stride != a.rows.q_out_stride)
        return bad(IDX_ERR_INVALID_ARG, "%s: q_out in place of q needs q's stride", what);
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.dk = dk;
    a.dv = dv;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.kc_stride = kc_stride;
    a.vc_stride = vc_stride;
    a.kv_rows = kv_rows;
    return cuda_status(launch_append(a, dtype, q4, geom_of(batch), st), what);
}

}  // namespace
}  // namespace lidx

using namespace lidx;

extern "C" {

idx_status idx_cache_append(const idx_new_rows* rows, idx_dtype dtype, int32_t n_q_heads, int32_t n_kv_heads,
                            int32_t dk, int32_t dv, idx_batch batch, const idx_rope* rope, void* k_cache,
                            int64_t k_row_stride, void* v_cache, int64_t v_row_stride, int64_t kv_rows,
                            idx_stream_t stream) {
    return append("idx_cache_append", false, rows, dtype, n_q_heads, n_kv_heads, dk, dv, batch, rope, k_cache, k_row_stride,
                  v_cache, v_row_stride, kv_rows, (cudaStream_t)stream);
}

idx_status idx_cache_append_q4(const idx_new_rows* rows, idx_dtype dtype, int32_t n_q_heads, int32_t n_kv_heads,
                               int32_t dk, int32_t dv, idx_batch batch, const idx_rope* rope, void* k_cache,
                               int64_t k_row_stride, void* v_cache, int64_t v_row_stride, int64_t kv_rows,
                               idx_stream_t stream) {
    return append("idx_cache_append_q4", true, rows, dtype, n_q_heads, n_kv_heads, dk, dv, batch, rope, k_cache, k_row_stride,
                  v_cache, v_row_stride, kv_rows, (cudaStream_t)stream);
}

size_t idx_q4_row_bytes(int32_t n_heads, int32_t d) {
    if (n_heads < 1 || d < 1 || d % 8) return 0;
    return (size_t)((q4_payload(n_heads, d) + 15) / 16 * 16);
}

idx_status idx_cache_read_q4(const void* k_cache, int64_t k_row_stride, const void* v_cache, int64_t v_row_stride,
                             int64_t kv_rows, int32_t n_kv_heads, int32_t dk, int32_t dv, idx_batch batch,
                             idx_dtype dtype, void* k_out, void* v_out, idx_stream_t stream) {
    const char* what = "idx_cache_read_q4";
    idx_status s = validate_batch(batch, what);
    if (s != IDX_OK) return s;
    if (!valid_dtype(dtype)) return bad(IDX_ERR_INVALID_ARG, "%s: bad dtype", what);
    if (n_kv_heads < 1 || dk < 1 || dk > 576 || dv < 0 || dv > 512 || dk % 8 || dv % 8)
        return bad(IDX_ERR_INVALID_ARG, "%s: need heads, and 1 <= dk <= 576, 0 <= dv <= 512 in multiples of 8", what);
    if ((int64_t)n_kv_heads * (dk + dv) > INT32_MAX / 2) return bad(IDX_ERR_UNSUPPORTED, "%s: rows too wide", what);
    if (kv_rows < 0) return bad(IDX_ERR_INVALID_ARG, "%s: kv_rows < 0", what);
    if (dv == 0 && (v_cache || v_out)) return bad(IDX_ERR_INVALID_ARG, "%s: v_cache and v_out need dv > 0", what);
    s = check_q4(what, "k_cache", k_cache, k_row_stride, n_kv_heads, dk);
    if (s == IDX_OK && dv) s = check_q4(what, "v_cache", v_cache, v_row_stride, n_kv_heads, dv);
    if (s != IDX_OK) return s;
    if ((int64_t)batch.n_seq * batch.n_q_per_seq == 0) return IDX_OK;
    if (!k_out || (dv && !v_out) || (kv_rows > 0 && (!k_cache || (dv && !v_cache))))
        return bad(IDX_ERR_INVALID_ARG, "%s: NULL caches or outputs", what);
    if (!aligned(k_out, 16) || !aligned(v_out, 16))
        return bad(IDX_ERR_INVALID_ARG, "%s: outputs must be 16-byte aligned", what);
    ReadArgs a = {};
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.kc_stride = k_row_stride;
    a.vc_stride = v_row_stride;
    a.kv_rows = kv_rows;
    a.Hkv = n_kv_heads;
    a.dk = dk;
    a.dv = dv;
    a.k_out = k_out;
    a.v_out = v_out;
    return cuda_status(launch_read_q4(a, dtype, geom_of(batch), (cudaStream_t)stream), what);
}

size_t dense_attn_q4_workspace_size(idx_dtype dtype, int32_t n_seq, int32_t n_q_per_seq, int32_t max_n_kv,
                                    int32_t n_q_heads, int32_t n_kv_heads, int32_t dk, int32_t dv) {
    if (!valid_dtype(dtype) || n_seq < 1 || n_q_per_seq < 1 || max_n_kv < 1 || n_kv_heads < 1 || n_q_heads < 1 ||
        n_q_heads % n_kv_heads || dk < 1 || dk > 576 || dv < 1 || dv > 512 || dk % 8 || dv % 8)
        return 0;
    return q4_attn_workspace_bytes(dtype, n_seq, n_q_per_seq, max_n_kv, n_q_heads, n_kv_heads, dk, dv);
}

idx_status dense_attn_q4(const void* q, idx_dtype dtype, int32_t n_q_heads, int32_t n_kv_heads, int32_t dk, int32_t dv,
                         const void* k_cache, int64_t k_row_stride, const void* v_cache, int64_t v_row_stride,
                         int64_t kv_rows, idx_batch batch, const idx_attn_mods* mods, float scale, void* out,
                         float* lse, void* workspace, size_t workspace_bytes, idx_stream_t stream) {
    const char* what = "dense_attn_q4";
    idx_status s = validate_batch(batch, what);
    if (s != IDX_OK) return s;
    if (!valid_dtype(dtype)) return bad(IDX_ERR_INVALID_ARG, "%s: bad dtype", what);
    if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads != 0)
        return bad(IDX_ERR_INVALID_ARG, "%s: need Hq, Hkv >= 1 and Hq %% Hkv == 0", what);
    if (dk < 1 || dk > 576 || dv < 1 || dv > 512 || dk % 8 || dv % 8)
        return bad(IDX_ERR_INVALID_ARG, "%s: need 1 <= dk <= 576 and 1 <= dv <= 512 in multiples of 8", what);
    if ((int64_t)n_kv_heads * (dk + dv) > INT32_MAX / 2) return bad(IDX_ERR_UNSUPPORTED, "%s: rows too wide", what);
    if (kv_rows < 0) return bad(IDX_ERR_INVALID_ARG, "%s: kv_rows < 0", what);
    s = check_q4(what, "k_cache", k_cache, k_row_stride, n_kv_heads, dk);
    if (s == IDX_OK) s = check_q4(what, "v_cache", v_cache, v_row_stride, n_kv_heads, dv);
    if (s != IDX_OK) return s;
    if (!(std::fabs(scale) <= 0x1p127f)) return bad(IDX_ERR_INVALID_ARG, "%s: scale not finite or above 2^127", what);
    DenseArgs a = {};
    if (mods) a.mods = *mods;
    if (!(a.mods.softcap >= 0.f && a.mods.softcap <= 0x1p127f))
        return bad(IDX_ERR_INVALID_ARG, "%s: softcap must be finite and >= 0, at most 2^127", what);
    if (a.mods.softcap > 0.f && !std::isfinite(scale / a.mods.softcap))
        return bad(IDX_ERR_INVALID_ARG, "%s: scale / softcap must be finite", what);
    if (a.mods.window < 0) return bad(IDX_ERR_INVALID_ARG, "%s: window < 0", what);
    if (!batch.q_pos && (a.mods.window > 0 || a.mods.slopes || a.mods.prefix_len || a.mods.prefix_end))
        return bad(IDX_ERR_INVALID_ARG, "%s: window, slopes, prefix_len and prefix_end need q_pos", what);
    if (!aligned(workspace, 16)) return bad(IDX_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", what);
    if (batch.max_n_kv > INT32_MAX - 1024)
        return bad(IDX_ERR_UNSUPPORTED, "%s: max_n_kv must be at most 2^31 - 1025", what);
    if ((int64_t)batch.n_seq * batch.n_q_per_seq == 0) return IDX_OK;
    if (!q || !out || (batch.max_n_kv > 0 && (!k_cache || !v_cache)))
        return bad(IDX_ERR_INVALID_ARG, "%s: NULL q, caches or out", what);
    a.q = q;
    a.Hq = n_q_heads;
    a.Hkv = n_kv_heads;
    a.dk = dk;
    a.dv = dv;
    a.k = k_cache;
    a.v = v_cache;
    a.k_stride = k_row_stride;
    a.v_stride = v_row_stride;
    a.kv_rows = kv_rows;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    return cuda_status(launch_attn_q4(a, dtype, geom_of(batch), workspace, workspace ? workspace_bytes : 0, (cudaStream_t)stream),
                       what);
}

size_t idx_beam_workspace_size(int32_t n_seq, int32_t n_beams, int32_t n_out, int32_t n_vocab) {
    if (n_seq < 1 || n_beams < 1 || n_out < 1 || n_out > kBeamOutMax || n_vocab < 1) return 0;
    return (size_t)beam_workspace_bytes(n_seq, n_beams, n_out, n_vocab);
}

idx_status idx_beam_step(const idx_beam* beam, idx_dtype dtype, int32_t n_seq, int32_t n_beams, int32_t n_out,
                         int32_t n_vocab, int32_t end_token, void* workspace, size_t workspace_bytes,
                         idx_stream_t stream) {
    const char* what = "idx_beam_step";
    if (!beam) return bad(IDX_ERR_INVALID_ARG, "%s: beam is NULL", what);
    if (!valid_dtype(dtype)) return bad(IDX_ERR_INVALID_ARG, "%s: bad dtype", what);
    if (n_seq < 0 || n_beams < 1 || n_vocab < 1) return bad(IDX_ERR_INVALID_ARG, "%s: need n_seq >= 0, n_beams, n_vocab >= 1", what);
    if (n_out < 1 || n_out > kBeamOutMax) return bad(IDX_ERR_INVALID_ARG, "%s: n_out must be in [1, %d]", what, kBeamOutMax);
    if ((int64_t)n_beams * n_vocab > INT32_MAX)
        return bad(IDX_ERR_INVALID_ARG, "%s: more than 2^31-1 continuations of a sequence", what);
    if ((int64_t)n_seq * n_beams > INT32_MAX || (int64_t)n_seq * n_out > INT32_MAX)
        return bad(IDX_ERR_INVALID_ARG, "%s: more than 2^31-1 rows", what);
    if (end_token < -1 || end_token >= n_vocab) return bad(IDX_ERR_INVALID_ARG, "%s: end_token outside [-1, n_vocab)", what);
    if (beam->done && end_token < 0) return bad(IDX_ERR_INVALID_ARG, "%s: done needs an end_token", what);
    if (beam->logit_stride < n_vocab) return bad(IDX_ERR_INVALID_ARG, "%s: logit_stride < n_vocab", what);
    if (beam->history_cols < 0 || (beam->lengths && (beam->history_stride < beam->history_cols ||
                                                     beam->out_history_stride < beam->history_cols)))
        return bad(IDX_ERR_INVALID_ARG, "%s: need 0 <= history_cols <= both histories' strides", what);
    if (n_beams > kBeamMax) return bad(IDX_ERR_UNSUPPORTED, "%s: n_beams > %d", what, kBeamMax);
    // (columns are counted in 32 bits up to the end of the last chunk)
    if (n_vocab > INT32_MAX - 65536) return bad(IDX_ERR_UNSUPPORTED, "%s: n_vocab > 2^31 - 65537", what);
    if (n_seq == 0) return IDX_OK;
    if (!beam->logits || !beam->scores || !beam->out_scores || !beam->parent || !beam->token || !beam->out_done)
        return bad(IDX_ERR_INVALID_ARG, "%s: NULL logits, scores or outputs", what);
    if (!beam->lengths != !beam->history || !beam->lengths != !beam->out_lengths || !beam->lengths != !beam->out_history)
        return bad(IDX_ERR_INVALID_ARG, "%s: lengths, history and their outputs come together", what);
    // outputs of n_out rows a sequence over inputs of n_beams rows a sequence: another sequence may still read them
    const int64_t in = (int64_t)n_seq * n_beams, out = (int64_t)n_seq * n_out;
    auto one = [](const void* p, int64_t n) -> Bytes { return {p, n, n, n}; };
    auto rows = [](const void* p, int64_t n, int64_t stride, int64_t cols, int64_t size) -> Bytes {
        return {p, cols ? ((n - 1) * stride + cols) * size : 0, stride * size, cols * size};
    };
    const Bytes reads[] = {rows(beam->logits, in, beam->logit_stride, n_vocab, dtype == IDX_F32 ? 4 : 2), one(beam->scores, 4 * in),
                           one(beam->done, in), one(beam->lengths, 4 * in),
                           rows(beam->history, in, beam->history_stride, beam->history_cols, 4)};
    const Bytes writes[] = {one(beam->out_scores, 4 * out), one(beam->parent, 4 * out), one(beam->token, 4 * out),
                            one(beam->out_done, out), one(beam->out_lengths, 4 * out),
                            rows(beam->out_history, out, beam->out_history_stride, beam->history_cols, 4)};
    for (const Bytes& w : writes)
        for (const Bytes& r : reads)
            if (overlap(w, r)) return bad(IDX_ERR_INVALID_ARG, "%s: an output overlaps an input", what);
    const size_t need = (size_t)beam_workspace_bytes(n_seq, n_beams, n_out, n_vocab);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
        return bad(IDX_ERR_INVALID_ARG, "%s: needs a 16-byte aligned workspace of %zu bytes (idx_beam_workspace_size)", what, need);
    return cuda_status(launch_beam(*beam, dtype, n_seq, n_beams, n_out, n_vocab, end_token, workspace, (cudaStream_t)stream),
                       what);
}

}  // extern "C"
