// lm_api.hip -- C interface of the language-model operators: argument checks and dispatch.
//
// Every check that needs no device data happens here, before anything is enqueued; the kernels
// never see an argument this file rejected.
#include <math.h>

#include "det_internal.h"

using namespace det;

namespace {

bool lm_dtype(det_dtype d) { return d == DET_F32 || d == DET_F16 || d == DET_BF16; }

bool aligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr double kMaxBytes = 4.6e18;      // 2^62

// [rows] rows of d elements, stride apart
struct Rows {
    const void* p;
    int64_t stride, rows, d;
    size_t es;

    bool ok() const {      // present, aligned, rows apart
        return p && aligned(p, es) && stride >= 0 && (rows <= 1 || stride >= d);
    }
    bool fits() const { return (double)rows * (double)(stride > d ? stride : d) * es < kMaxBytes; }
    size_t bytes() const {
        return rows > 0 && d > 0 ? ((size_t)(rows - 1) * stride + d) * es : 0;
    }
};

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && an > 0 && bn > 0 && x < y + bn && y < x + an;
}

// `out` (contiguous) lies apart from `in`, or is the very same rows when in_place allows that
bool apart(const Rows& in, const Rows& out, bool in_place) {
    if (in_place && in.p == out.p && (in.stride == out.stride || in.rows <= 1)) return true;
    return !overlap(in.p, in.bytes(), out.p, out.bytes());
}

bool apart(const void* a, size_t an, const Rows& r) { return !overlap(a, an, r.p, r.bytes()); }

det_status ws_status(const void* ws, size_t ws_bytes, size_t need) {
    return ws && aligned(ws, 256) && ws_bytes >= need ? DET_SUCCESS : DET_ERROR_WORKSPACE;
}

}  // namespace

extern "C" {

det_status det_rms_norm(const void* x, int64_t x_stride, const void* residual,
                        int64_t residual_stride, const void* weight, int64_t rows, int64_t d,
                        det_dtype dtype, double eps, void* h, void* y, det_dtype y_dtype,
                        int64_t group, float* scales, float* rstd, void* stream) {
    if (!lm_dtype(dtype)) return DET_ERROR_UNSUPPORTED;
    const bool codes = y_dtype == DET_E4M3;
    if (!codes && y_dtype != dtype) return DET_ERROR_UNSUPPORTED;
    if (rows < 0 || d < 0 || !(eps >= 0.0) || !isfinite((float)eps))
        return DET_ERROR_INVALID_VALUE;
    if (rows > DET_MAX_N || d > DET_MAX_N) return DET_ERROR_TOO_LARGE;
    if (codes ? group != 0 && group != 32 && group != 64 && group != 128 : group != 0)
        return DET_ERROR_INVALID_VALUE;
    if (rows == 0) return DET_SUCCESS;
    if (d == 0) return DET_ERROR_INVALID_VALUE;
    const size_t es = lm_size(dtype);
    const Rows in{x, x_stride, rows, d, es}, res{residual, residual_stride, rows, d, es};
    const Rows ho{h, d, rows, d, es}, yo{y, d, rows, d, lm_size(y_dtype)};
    if (!in.ok() || !yo.ok() || !weight || !aligned(weight, es)) return DET_ERROR_INVALID_VALUE;
    if (residual ? !res.ok() || !ho.ok() : h != nullptr) return DET_ERROR_INVALID_VALUE;
    if (!in.fits() || !yo.fits() || (residual && !res.fits())) return DET_ERROR_TOO_LARGE;
    if (codes ? !scales || !aligned(scales, 4) : scales != nullptr) return DET_ERROR_INVALID_VALUE;
    if (rstd && !aligned(rstd, 4)) return DET_ERROR_INVALID_VALUE;
    // what is written lies apart from what is read and from each other; h may replace an input
    const size_t wbytes = (size_t)d * es, sbytes = (size_t)rows * 4;
    const size_t cbytes = codes ? sbytes * (group ? (d + group - 1) / group : 1) : 0;
    if (!apart(in, yo, false) || !apart(weight, wbytes, yo) ||
        overlap(scales, cbytes, rstd, sbytes) || overlap(scales, cbytes, weight, wbytes) ||
        overlap(rstd, sbytes, weight, wbytes))
        return DET_ERROR_INVALID_VALUE;
    if (residual && (!apart(res, yo, false) || !apart(in, ho, true) || !apart(res, ho, true) ||
                     !apart(weight, wbytes, ho) || !apart(ho, yo, false)))
        return DET_ERROR_INVALID_VALUE;
    for (const Rows* r : {&in, &res, &ho, &yo})
        if (r->p && (!apart(scales, cbytes, *r) || !apart(rstd, sbytes, *r)))
            return DET_ERROR_INVALID_VALUE;
    const NormCall c{x, residual, weight, h, y, scales, rstd, x_stride, residual_stride,
                     rows, d, group, (float)eps, dtype, codes};
    return norm_launch(c, static_cast<hipStream_t>(stream));
}

size_t det_rms_norm_backward_workspace_size(int64_t rows, int64_t d, det_dtype dtype) {
    if (rows < 0 || rows > DET_MAX_N || d < 0 || d > DET_MAX_N || !lm_dtype(dtype)) return 0;
    return norm_backward_workspace(rows, d, dtype);
}

det_status det_rms_norm_backward(const void* dy, int64_t dy_stride, const void* h,
                                 int64_t h_stride, const void* weight, const float* rstd,
                                 const void* dh, int64_t dh_stride, int64_t rows, int64_t d,
                                 det_dtype dtype, void* dx, void* dweight, void* ws,
                                 size_t ws_bytes, void* stream) {
    if (!lm_dtype(dtype)) return DET_ERROR_UNSUPPORTED;
    if (rows < 0 || d < 0) return DET_ERROR_INVALID_VALUE;
    if (rows > DET_MAX_N || d > DET_MAX_N) return DET_ERROR_TOO_LARGE;
    if (d == 0) return rows == 0 ? DET_SUCCESS : DET_ERROR_INVALID_VALUE;
    const size_t es = lm_size(dtype);
    const Rows a{dy, dy_stride, rows, d, es}, b{h, h_stride, rows, d, es};
    const Rows e{dh, dh_stride, rows, d, es}, o{dx, d, rows, d, es};
    if (!dweight || !aligned(dweight, es)) return DET_ERROR_INVALID_VALUE;
    const size_t wbytes = (size_t)d * es;
    if (rows > 0) {
        if (!a.ok() || !b.ok() || !o.ok() || !weight || !aligned(weight, es) || !rstd ||
            !aligned(rstd, 4) || (dh && !e.ok()))
            return DET_ERROR_INVALID_VALUE;
        if (!a.fits() || !b.fits() || !o.fits() || (dh && !e.fits())) return DET_ERROR_TOO_LARGE;
        // rows beyond the registers are read twice, once more for the weight's sums
        const bool in_place = d <= 16384;
        if (!apart(a, o, in_place) || !apart(b, o, in_place) || (dh && !apart(e, o, in_place)) ||
            !apart(weight, wbytes, o) || !apart(rstd, (size_t)rows * 4, o))
            return DET_ERROR_INVALID_VALUE;
        for (const Rows* r : {&a, &b, &e, &o})
            if (r->p && !apart(dweight, wbytes, *r)) return DET_ERROR_INVALID_VALUE;
        if (overlap(weight, wbytes, dweight, wbytes) ||
            overlap(rstd, (size_t)rows * 4, dweight, wbytes))
            return DET_ERROR_INVALID_VALUE;
    }
    const det_status st = ws_status(ws, ws_bytes, norm_backward_workspace(rows, d, dtype));
    if (st != DET_SUCCESS) return st;
    const NormBackCall c{dy, h, weight, dh, rstd, dx, dweight, dy_stride, h_stride, dh_stride,
                         rows, d, dtype};
    return norm_backward_launch(c, ws, static_cast<hipStream_t>(stream));
}

}  // extern "C"

namespace {

// Checks what both directions share and fills the call; `t`: scores or dout.
det_status bias_checked(int64_t num_buckets, int64_t heads, int64_t max_distance, unsigned flags,
                        int64_t batch, int64_t q, int64_t k, int64_t q_offset,
                        const int32_t* q_offsets, const int32_t* lengths, const void* t,
                        int64_t stride_b, int64_t stride_h, int64_t stride_q, det_dtype dtype,
                        BiasCall* c) {
    if (!lm_dtype(dtype)) return DET_ERROR_UNSUPPORTED;
    if (flags & ~(DET_BIAS_BIDIRECTIONAL | DET_BIAS_CAUSAL)) return DET_ERROR_INVALID_VALUE;
    if (batch < 0 || q < 0 || k < 0 || heads < 1 || num_buckets < 1) return DET_ERROR_INVALID_VALUE;
    if (num_buckets > DET_BIAS_MAX_BUCKETS || heads > 65535 || batch > DET_MAX_N ||
        q > DET_MAX_N || k > DET_MAX_N || max_distance > DET_MAX_N)
        return DET_ERROR_TOO_LARGE;
    const bool both = flags & DET_BIAS_BIDIRECTIONAL;
    const int64_t side = both ? num_buckets / 2 : num_buckets;
    if (side > kBiasMaxSide) return DET_ERROR_TOO_LARGE;
    if (side < 2 || max_distance <= side / 2) return DET_ERROR_INVALID_VALUE;
    if (q_offset > (1LL << 40) || q_offset < -(1LL << 40)) return DET_ERROR_INVALID_VALUE;
    if (!aligned(q_offsets, 4) || !aligned(lengths, 4)) return DET_ERROR_INVALID_VALUE;
    const size_t es = lm_size(dtype);
    if ((double)batch * heads * (double)q * (double)k * es > kMaxBytes) return DET_ERROR_TOO_LARGE;
    if (t) {
        if (!aligned(t, es) || stride_b < 0 || stride_h < 0 || stride_q < 0)
            return DET_ERROR_INVALID_VALUE;
        if (((double)batch * stride_b + (double)heads * stride_h + (double)q * stride_q + k) * es >
            kMaxBytes)
            return DET_ERROR_TOO_LARGE;
    }
    *c = BiasCall{nullptr, t, nullptr, stride_b, stride_h, stride_q, batch, heads, q, k, q_offset,
                  max_distance, q_offsets, lengths, (int)num_buckets, both,
                  (flags & DET_BIAS_CAUSAL) != 0, -INFINITY, dtype};
    return DET_SUCCESS;
}

size_t strided_bytes(const BiasCall& c) {
    return ((size_t)(c.batch - 1) * c.sb + (size_t)(c.heads - 1) * c.sh +
            (size_t)(c.q - 1) * c.sq + c.k) * lm_size(c.dtype);
}

bool contiguous(const BiasCall& c) {
    return (c.sq == c.k || c.q == 1) && (c.sh == c.q * c.k || c.heads == 1) &&
           (c.sb == c.heads * c.q * c.k || c.batch == 1);
}

// `out` may be the call's own strided tensor where that is contiguous, else lies apart from it;
// and from the masks' arguments, which every workgroup reads
bool bias_out_ok(const BiasCall& c, const void* out, size_t obytes) {
    if (!out || !aligned(out, lm_size(c.dtype)) ||
        overlap(out, obytes, c.q_offsets, (size_t)c.batch * 4) ||
        overlap(out, obytes, c.lengths, (size_t)c.batch * 4))
        return false;
    if (!c.scores || (out == c.scores && contiguous(c))) return true;
    return !overlap(out, obytes, c.scores, strided_bytes(c));
}

}  // namespace

extern "C" {

det_status det_relative_bias(const void* table, int64_t num_buckets, int64_t heads,
                             int64_t max_distance, unsigned flags, int64_t batch, int64_t q,
                             int64_t k, int64_t q_offset, const int32_t* q_offsets,
                             const int32_t* lengths, const void* scores, int64_t stride_b,
                             int64_t stride_h, int64_t stride_q, det_dtype dtype, void* out,
                             void* stream) {
    BiasCall c;
    const det_status st = bias_checked(num_buckets, heads, max_distance, flags, batch, q, k,
                                       q_offset, q_offsets, lengths, scores, stride_b, stride_h,
                                       stride_q, dtype, &c);
    if (st != DET_SUCCESS) return st;
    if (batch == 0 || q == 0 || k == 0) return DET_SUCCESS;
    const size_t es = lm_size(dtype), obytes = (size_t)batch * heads * q * k * es;
    if (!table || !aligned(table, es) || !bias_out_ok(c, out, obytes) ||
        overlap(out, obytes, table, (size_t)num_buckets * heads * es))
        return DET_ERROR_INVALID_VALUE;
    c.table = table;
    c.out = out;
    return bias_launch(c, static_cast<hipStream_t>(stream));
}

size_t det_relative_bias_backward_workspace_size(int64_t batch, int64_t heads, int64_t q,
                                                 int64_t k, int64_t num_buckets, det_dtype dtype) {
    if (!lm_dtype(dtype) || batch < 0 || batch > DET_MAX_N || heads < 1 || heads > 65535 || q < 0 ||
        q > DET_MAX_N || k < 0 || k > DET_MAX_N || num_buckets < 1 ||
        num_buckets > DET_BIAS_MAX_BUCKETS ||
        (double)batch * heads * (double)q * (double)k * lm_size(dtype) > kMaxBytes)
        return 0;
    return bias_backward_workspace(batch, heads, q, k, (int)num_buckets, dtype);
}

det_status det_relative_bias_backward(const void* dout, int64_t stride_b, int64_t stride_h,
                                      int64_t stride_q, int64_t num_buckets, int64_t heads,
                                      int64_t max_distance, unsigned flags, int64_t batch,
                                      int64_t q, int64_t k, int64_t q_offset,
                                      const int32_t* q_offsets, const int32_t* lengths,
                                      det_dtype dtype, void* dtable, void* dscores, void* ws,
                                      size_t ws_bytes, void* stream) {
    BiasCall c;
    det_status st = bias_checked(num_buckets, heads, max_distance, flags, batch, q, k, q_offset,
                                 q_offsets, lengths, dout, stride_b, stride_h, stride_q, dtype, &c);
    if (st != DET_SUCCESS) return st;
    const size_t es = lm_size(dtype), obytes = (size_t)batch * heads * q * k * es;
    const size_t tbytes = (size_t)num_buckets * heads * es;
    if (!dtable || !aligned(dtable, es)) return DET_ERROR_INVALID_VALUE;
    if (obytes > 0 &&
        (!dout || overlap(dtable, tbytes, dout, strided_bytes(c)) ||
         overlap(dtable, tbytes, q_offsets, (size_t)batch * 4) ||
         overlap(dtable, tbytes, lengths, (size_t)batch * 4) ||
         (dscores && (!bias_out_ok(c, dscores, obytes) || overlap(dscores, obytes, dtable, tbytes)))))
        return DET_ERROR_INVALID_VALUE;
    st = ws_status(ws, ws_bytes, bias_backward_workspace(batch, heads, q, k, (int)num_buckets, dtype));
    if (st != DET_SUCCESS) return st;
    st = bias_backward_launch(c, dout, dtable, ws, static_cast<hipStream_t>(stream));
    if (st != DET_SUCCESS || !dscores || obytes == 0) return st;
    c.out = dscores;
    c.fill = 0.0f;
    return bias_launch(c, static_cast<hipStream_t>(stream));
}

det_status det_token_logprobs(const void* logits, int64_t row_stride, const int64_t* targets,
                              int64_t rows, int64_t vocab, det_dtype dtype, double scale,
                              float* logp, float* entropy, float* lse, int64_t top,
                              float* top_logp, int64_t* top_ids, void* stream) {
    if (!lm_dtype(dtype)) return DET_ERROR_UNSUPPORTED;
    if (rows < 0 || vocab < 0 || top < 0 || !((float)scale > 0.0f) || !isfinite((float)scale))
        return DET_ERROR_INVALID_VALUE;
    if (rows > DET_MAX_N || vocab > DET_MAX_N) return DET_ERROR_TOO_LARGE;
    if (top > vocab || top > DET_LOGPROB_MAX_TOP) return DET_ERROR_INVALID_VALUE;
    if (top > 0 && vocab > DET_LOGPROB_MAX_TOP_VOCAB) return DET_ERROR_TOO_LARGE;
    if (rows == 0) return DET_SUCCESS;
    const Rows in{logits, row_stride, rows, vocab, lm_size(dtype)};
    if (vocab == 0 || !in.ok() || !targets || !aligned(targets, 8)) return DET_ERROR_INVALID_VALUE;
    if (!in.fits()) return DET_ERROR_TOO_LARGE;
    if (!logp || !entropy || !lse ||
        (top > 0 ? !top_logp || !top_ids || !aligned(top_ids, 8) : top_logp || top_ids))
        return DET_ERROR_INVALID_VALUE;
    // what is written lies apart from what is read and from each other
    const struct { const void* p; size_t bytes; } outs[] = {
        {logp, (size_t)rows * 4}, {entropy, (size_t)rows * 4}, {lse, (size_t)rows * 4},
        {top_logp, (size_t)rows * top * 4}, {top_ids, (size_t)rows * top * 8}};
    for (const auto& o : outs) {
        if (!aligned(o.p, 4) || !apart(o.p, o.bytes, in) ||
            overlap(o.p, o.bytes, targets, (size_t)rows * 8))
            return DET_ERROR_INVALID_VALUE;
        for (const auto& other : outs)
            if (&o != &other && overlap(o.p, o.bytes, other.p, other.bytes))
                return DET_ERROR_INVALID_VALUE;
    }
    const LogpCall c{logits, targets, logp, entropy, lse, top_logp, top_ids, row_stride, rows,
                     vocab, (int)top, (float)scale, dtype};
    return logprob_launch(c, static_cast<hipStream_t>(stream));
}

det_status det_token_logprobs_backward(const void* logits, int64_t row_stride,
                                       const int64_t* targets, const float* lse,
                                       const float* dlogp, const float* entropy,
                                       const float* dentropy, int64_t rows, int64_t vocab,
                                       det_dtype dtype, double scale, void* dlogits,
                                       int64_t dlogits_stride, void* stream) {
    if (!lm_dtype(dtype)) return DET_ERROR_UNSUPPORTED;
    if (rows < 0 || vocab < 0 || !((float)scale > 0.0f) || !isfinite((float)scale))
        return DET_ERROR_INVALID_VALUE;
    if (rows > DET_MAX_N || vocab > DET_MAX_N) return DET_ERROR_TOO_LARGE;
    if (rows == 0) return DET_SUCCESS;
    const size_t es = lm_size(dtype);
    const Rows in{logits, row_stride, rows, vocab, es}, out{dlogits, dlogits_stride, rows, vocab, es};
    if (vocab == 0 || !in.ok() || !out.ok() || !targets || !aligned(targets, 8))
        return DET_ERROR_INVALID_VALUE;
    if (!in.fits() || !out.fits()) return DET_ERROR_TOO_LARGE;
    if (!lse || !dlogp || (dentropy && !entropy)) return DET_ERROR_INVALID_VALUE;
    for (const void* p : {(const void*)lse, (const void*)dlogp, (const void*)entropy,
                          (const void*)dentropy})
        if (p && (!aligned(p, 4) || !apart(p, (size_t)rows * 4, out)))
            return DET_ERROR_INVALID_VALUE;
    if (!apart(in, out, true) || !apart(targets, (size_t)rows * 8, out))
        return DET_ERROR_INVALID_VALUE;
    const LogpBackCall c{logits, targets, lse, dlogp, entropy, dentropy, dlogits, row_stride,
                         dlogits_stride, rows, vocab, (float)scale, dtype};
    return logprob_backward_launch(c, static_cast<hipStream_t>(stream));
}

}  // extern "C"
