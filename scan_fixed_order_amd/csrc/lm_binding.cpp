// lm_binding.cpp -- the language-model operators' binding: torch tensors in, device pointers out.
//
// Argument marshalling only, like the ctypes binding of the other operations, in C++ because the
// calls are small: a norm of one token runs for 3 us on the GPU, and checking five tensors and
// allocating three outputs from Python takes 9.  Outputs and workspaces come from torch's caching
// allocator, the work goes to torch's current stream.
#include <ATen/ATen.h>
#include <ATen/hip/HIPContext.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>

#include "det.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Optional = std::optional<Tensor>;

[[noreturn]] void wrong_type(const std::string& what) { throw py::type_error(what); }
[[noreturn]] void wrong_value(const std::string& what) { throw py::value_error(what); }

void check_status(det_status st, const char* what) {
    if (st == DET_SUCCESS) return;
    const py::object error = py::module_::import("scan_fixed_order_amd.det").attr("DetError");
    PyErr_SetObject(error.ptr(), error((int)st, what).ptr());
    throw py::error_already_set();
}

det_dtype lm_type(const Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return DET_F32;
        case at::kHalf: return DET_F16;
        case at::kBFloat16: return DET_BF16;
        default:
            wrong_type(std::string("the language-model operators take float32, float16 and "
                                   "bfloat16, got ") + c10::toString(t.scalar_type()));
    }
}

void same_type(const Tensor& t, const Tensor& like, const char* what) {
    if (t.scalar_type() != like.scalar_type())
        wrong_type(std::string(what) + " must be " + c10::toString(like.scalar_type()) + ", got " +
                   c10::toString(t.scalar_type()));
}

// device, type, shape and contiguity of an argument
const Tensor& of(const Tensor& t, at::ScalarType type, at::IntArrayRef shape, const char* what) {
    if (t.scalar_type() != type)
        wrong_type(std::string(what) + " must be " + c10::toString(type) + ", got " +
                   c10::toString(t.scalar_type()));
    if (t.sizes() != shape) wrong_value(std::string(what) + " has the wrong shape");
    if (!t.is_contiguous())
        wrong_value(std::string("det needs contiguous tensors (") + what +
                    "; views with an offset are fine)");
    return t;
}

void* pointer(const Tensor& t, const Tensor& first) {
    if (!t.is_cuda()) wrong_value("det operates on device tensors");
    if (t.get_device() != first.get_device()) wrong_value("det needs tensors of one device");
    return t.data_ptr();
}

void* pointer(const Optional& t, const Tensor& first) {
    return t ? pointer(*t, first) : nullptr;
}

// Elements between neighbouring rows (the last dimension is a row): the leading dimensions have
// to collapse into one.
int64_t row_stride(const Tensor& t, const char* what) {
    const int64_t n = t.size(-1);
    if (t.is_contiguous()) return n;
    if (t.stride(-1) == 1 || n == 1) {
        int64_t stride = -1, span = 0;
        bool even = true;
        for (int64_t i = t.dim() - 2; i >= 0 && even; --i) {
            const int64_t size = t.size(i), st = t.stride(i);
            if (size == 1) continue;
            if (stride < 0)
                stride = st;
            else
                even = st == span;
            span = st * size;
        }
        if (even && stride < 0) return n;
        if (even && stride >= n) return stride;
    }
    wrong_value(std::string("det needs the rows of ") + what + " contiguous and evenly spaced");
}

Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
    return at::empty(shape, like.options().dtype(type));
}

Tensor workspace(size_t bytes, const Optional& ws, const Tensor& like) {
    if (!ws) return empty({(int64_t)(bytes < 256 ? 256 : bytes)}, at::kByte, like);
    if (ws->nbytes() < bytes)
        wrong_value("workspace of " + std::to_string(bytes) + " bytes needed");
    return *ws;
}

// An expanded view has more bytes than memory: checked before any size is trusted.
void check_workspace(const Optional& ws) {
    if (ws && !ws->is_contiguous()) wrong_value("a workspace must be contiguous");
}

// the device of `t` while the call lasts
using Guard = c10::DeviceGuard;

void* stream(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.get_device()).stream(); }

// Number of rows (the last dimension is a row).  From the leading dimensions, not numel(): rows of
// no elements are rows, and the library refuses them.
int64_t rows_of(const Tensor& t, const char* what) {
    if (t.dim() < 1) wrong_value(std::string(what) + " must have at least one dimension");
    return c10::multiply_integers(t.sizes().slice(0, t.dim() - 1));
}

// ---------------------------------------------------------------- norm

py::tuple rms_norm(const Tensor& x, const Tensor& weight, double eps, const Optional& residual,
                   bool codes, int64_t group) {
    const det_dtype type = lm_type(x);
    const int64_t rows = rows_of(x, "x"), d = x.size(-1);
    const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
    of(weight, x.scalar_type(), {d}, "weight");
    const int64_t stride = row_stride(x, "x");
    int64_t res_stride = 0;
    if (residual) {
        same_type(*residual, x, "residual");
        if (residual->sizes() != x.sizes()) wrong_value("residual must have the shape of x");
        res_stride = row_stride(*residual, "residual");
    }
    if (codes) {
        if (group != 0 && group != 32 && group != 64 && group != 128)
            wrong_value("group must be 0, 32, 64 or 128");
    } else if (group) {
        wrong_value("group is for an 8-bit output");
    }
    void* const xp = pointer(x, x);
    void* const rp = pointer(residual, x);
    void* const wp = pointer(weight, x);
    const Guard guard(x.device());
    Tensor h, scales;
    if (residual) h = empty(x.sizes(), x.scalar_type(), x);
    if (codes) {
        at::DimVector shape(lead.begin(), lead.end());
        shape.push_back(group ? (d + group - 1) / group : 1);
        scales = empty(shape, at::kFloat, x);
    }
    const Tensor y = empty(x.sizes(), codes ? at::kFloat8_e4m3fn : x.scalar_type(), x);
    const Tensor rstd = empty(lead, at::kFloat, x);
    check_status(det_rms_norm(xp, stride, rp, res_stride, wp, rows, d, type, eps,
                              residual ? h.data_ptr() : nullptr, y.data_ptr(),
                              codes ? DET_E4M3 : type, group,
                              codes ? scales.data_ptr<float>() : nullptr, rstd.data_ptr<float>(),
                              stream(x)),
                 "det_rms_norm");
    return py::make_tuple(y, residual ? h : x, rstd,
                          codes ? py::cast(scales) : py::object(py::none()));
}

py::tuple rms_norm_backward(const Tensor& dy, const Tensor& h, const Tensor& weight,
                            const Tensor& rstd, const Optional& dh, const Optional& ws) {
    const det_dtype type = lm_type(h);
    const int64_t rows = rows_of(h, "h"), d = h.size(-1);
    of(weight, h.scalar_type(), {d}, "weight");
    of(rstd, at::kFloat, h.sizes().slice(0, h.dim() - 1), "rstd");
    same_type(dy, h, "dy");
    if (dy.sizes() != h.sizes()) wrong_value("dy must have the shape of h");
    if (dh) {
        same_type(*dh, h, "dh");
        if (dh->sizes() != h.sizes()) wrong_value("dh must have the shape of h");
    }
    check_workspace(ws);
    void* const dyp = pointer(dy, h);
    void* const hp = pointer(h, h);
    void* const wp = pointer(weight, h);
    void* const sp = pointer(rstd, h);
    void* const dhp = pointer(dh, h);
    const Guard guard(h.device());
    const Tensor dx = empty(h.sizes(), h.scalar_type(), h);
    const Tensor dweight = empty({d}, h.scalar_type(), h);
    const Tensor w = workspace(det_rms_norm_backward_workspace_size(rows, d, type), ws, h);
    check_status(det_rms_norm_backward(dyp, row_stride(dy, "dy"), hp, row_stride(h, "h"), wp,
                                       static_cast<const float*>(sp), dhp,
                                       dh ? row_stride(*dh, "dh") : 0, rows, d, type,
                                       dx.data_ptr(), dweight.data_ptr(), pointer(w, h),
                                       w.nbytes(), stream(h)),
                 "det_rms_norm_backward");
    return py::make_tuple(dx, dweight);
}

// ---------------------------------------------------------------- relative position bias

// The masks' arguments: a batch of -1 is not known yet.
int64_t bias_batch(int64_t batch, const Optional& offsets, const Optional& lengths) {
    const auto one = [&](const Optional& t, const char* what) {
        if (!t) return;
        if (t->dim() != 1) wrong_value(std::string(what) + " must be one-dimensional");
        if (batch < 0) batch = t->size(0);
        of(*t, at::kInt, {batch}, what);
    };
    one(offsets, "q_offset");
    one(lengths, "lengths");
    return batch < 0 ? 1 : batch;
}

void bias_strided(const Tensor& t, const char* what) {
    if (t.dim() != 4) wrong_value(std::string(what) + " must be [batch, heads, q, k]");
    if (t.stride(3) != 1 && t.size(3) > 1)
        wrong_value(std::string("det needs the rows of ") + what + " contiguous");
}

Tensor relative_bias(const Tensor& table, int64_t q, int64_t k, const Optional& scores,
                     int64_t max_distance, unsigned flags, int64_t offset, const Optional& offsets,
                     const Optional& lengths, const Optional& out) {
    const det_dtype type = lm_type(table);
    if (table.dim() != 2) wrong_value("table must be [buckets, heads]");
    if (q < 0 || k < 0) wrong_value("q and k must not be negative");
    of(table, table.scalar_type(), table.sizes(), "table");
    const int64_t buckets = table.size(0), heads = table.size(1);
    int64_t batch = -1, sb = 0, sh = 0, sq = 0;
    if (scores) {
        same_type(*scores, table, "scores");
        bias_strided(*scores, "scores");
        batch = scores->size(0);
        if (scores->size(1) != heads || scores->size(2) != q || scores->size(3) != k)
            wrong_value("scores must be [batch, heads, q, k]");
        sb = scores->stride(0);
        sh = scores->stride(1);
        sq = scores->stride(2);
    }
    batch = bias_batch(batch, offsets, lengths);
    if (out) of(*out, table.scalar_type(), {batch, heads, q, k}, "out");
    void* const tp = pointer(table, table);
    void* const sp = pointer(scores, table);
    void* const op = pointer(offsets, table);
    void* const lp = pointer(lengths, table);
    const Guard guard(table.device());
    const Tensor o = out ? *out : empty({batch, heads, q, k}, table.scalar_type(), table);
    check_status(det_relative_bias(tp, buckets, heads, max_distance, flags, batch, q, k, offset,
                                   static_cast<const int32_t*>(op), static_cast<const int32_t*>(lp),
                                   sp, sb, sh, sq, type, pointer(o, table), stream(table)),
                 "det_relative_bias");
    return o;
}

Tensor relative_bias_backward(const Tensor& dout, int64_t buckets, int64_t max_distance,
                              unsigned flags, int64_t offset, const Optional& offsets,
                              const Optional& lengths, const Optional& dscores, const Optional& ws) {
    const det_dtype type = lm_type(dout);
    bias_strided(dout, "dout");
    if (buckets < 0) wrong_value("num_buckets must not be negative");
    const int64_t batch = dout.size(0), heads = dout.size(1), q = dout.size(2), k = dout.size(3);
    bias_batch(batch, offsets, lengths);
    if (dscores) of(*dscores, dout.scalar_type(), dout.sizes(), "dscores");
    check_workspace(ws);
    void* const dp = pointer(dout, dout);
    void* const op = pointer(offsets, dout);
    void* const lp = pointer(lengths, dout);
    const Guard guard(dout.device());
    const Tensor dtable = empty({buckets, heads}, dout.scalar_type(), dout);
    const Tensor w = workspace(
        det_relative_bias_backward_workspace_size(batch, heads, q, k, buckets, type), ws, dout);
    check_status(det_relative_bias_backward(dp, dout.stride(0), dout.stride(1), dout.stride(2),
                                            buckets, heads, max_distance, flags, batch, q, k,
                                            offset, static_cast<const int32_t*>(op),
                                            static_cast<const int32_t*>(lp), type,
                                            dtable.data_ptr(), pointer(dscores, dout),
                                            pointer(w, dout), w.nbytes(), stream(dout)),
                 "det_relative_bias_backward");
    return dtable;
}

// ---------------------------------------------------------------- token log probabilities

py::tuple token_logprobs(const Tensor& logits, const Tensor& targets, double scale, int64_t top) {
    const det_dtype type = lm_type(logits);
    rows_of(logits, "logits");
    if (top < 0 || top > DET_LOGPROB_MAX_TOP)
        wrong_value("top must lie in 0 .. " + std::to_string(DET_LOGPROB_MAX_TOP));
    const at::IntArrayRef shape = logits.sizes().slice(0, logits.dim() - 1);
    const int64_t vocab = logits.size(-1);
    of(targets, at::kLong, shape, "targets");
    const int64_t stride = row_stride(logits, "logits"), rows = targets.numel();
    void* const lp = pointer(logits, logits);
    void* const tp = pointer(targets, logits);
    const Guard guard(logits.device());
    const Tensor logp = empty(shape, at::kFloat, logits);
    const Tensor entropy = empty(shape, at::kFloat, logits);
    const Tensor lse = empty(shape, at::kFloat, logits);
    Tensor top_logp, top_ids;
    if (top) {
        at::DimVector wide(shape.begin(), shape.end());
        wide.push_back(top);
        top_logp = empty(wide, at::kFloat, logits);
        top_ids = empty(wide, at::kLong, logits);
    }
    check_status(det_token_logprobs(lp, stride, static_cast<const int64_t*>(tp), rows, vocab, type,
                                    scale, logp.data_ptr<float>(), entropy.data_ptr<float>(),
                                    lse.data_ptr<float>(), top,
                                    top ? top_logp.data_ptr<float>() : nullptr,
                                    top ? top_ids.data_ptr<int64_t>() : nullptr, stream(logits)),
                 "det_token_logprobs");
    if (!top) return py::make_tuple(logp, entropy, lse, py::none(), py::none());
    return py::make_tuple(logp, entropy, lse, top_logp, top_ids);
}

Tensor token_logprobs_backward(const Tensor& logits, const Tensor& targets, const Tensor& lse,
                               const Tensor& dlogp, const Optional& entropy,
                               const Optional& dentropy, double scale, const Optional& out) {
    const det_dtype type = lm_type(logits);
    const int64_t rows = rows_of(logits, "logits"), vocab = logits.size(-1);
    const at::IntArrayRef shape = logits.sizes().slice(0, logits.dim() - 1);
    of(targets, at::kLong, shape, "targets");
    of(lse, at::kFloat, shape, "lse");
    of(dlogp, at::kFloat, shape, "dlogp");
    if (entropy) of(*entropy, at::kFloat, shape, "entropy");
    if (dentropy) {
        of(*dentropy, at::kFloat, shape, "dentropy");
        if (!entropy) wrong_value("dentropy needs entropy");
    }
    const int64_t stride = row_stride(logits, "logits");
    if (out) {
        same_type(*out, logits, "out");
        if (out->sizes() != logits.sizes()) wrong_value("out must have the shape of logits");
    }
    void* const xp = pointer(logits, logits);
    void* const tp = pointer(targets, logits);
    void* const lp = pointer(lse, logits);
    void* const dp = pointer(dlogp, logits);
    void* const ep = pointer(entropy, logits);
    void* const dep = pointer(dentropy, logits);
    const Guard guard(logits.device());
    const Tensor o = out ? *out : empty(logits.sizes(), logits.scalar_type(), logits);
    check_status(det_token_logprobs_backward(
                     xp, stride, static_cast<const int64_t*>(tp), static_cast<const float*>(lp),
                     static_cast<const float*>(dp), static_cast<const float*>(ep),
                     static_cast<const float*>(dep), rows, vocab, type, scale,
                     pointer(o, logits), row_stride(o, "out"), stream(logits)),
                 "det_token_logprobs_backward");
    return o;
}

}  // namespace

PYBIND11_MODULE(_lm_binding, m) {
    m.def("row_stride", [](const Tensor& t, const std::string& what) {
        return row_stride(t, what.c_str());
    });
    m.def("rms_norm", &rms_norm);
    m.def("rms_norm_backward", &rms_norm_backward);
    m.def("relative_bias", &relative_bias);
    m.def("relative_bias_backward", &relative_bias_backward);
    m.def("token_logprobs", &token_logprobs);
    m.def("token_logprobs_backward", &token_logprobs_backward);
}
