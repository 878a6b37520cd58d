// torch_ops.cpp -- the norm and feed-forward calls of the Python binding that a
// step makes between launches: their checks, their allocations and the two
// autograd functions, in C++ over the C ABI of libfp8q (fp8q.h).  A small
// training step is bound by the host: forward and backward of a 16 x 256 norm
// through autograd take 57 us here and took 102 us with the functions in
// Python over ctypes, where a bare product and its gradient take 51.
//
// Raises ValueError and TypeError as the rest of the binding, and Fp8qError for
// a status other than 0 (a RuntimeError with the same text out of a backward
// pass, which runs on another thread).
#include <ATen/cuda/CUDAContext.h>
#include <ATen/cuda/EmptyTensor.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/extension.h>

#include <array>
#include <optional>
#include <sstream>

#include "fp8q.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using MaybeTensor = std::optional<Tensor>;

// ---------------------------------------------------------------------------
// checks, with the words of the binding's own
// ---------------------------------------------------------------------------
template <typename... Parts>
std::string text(const Parts&... parts) {
    std::ostringstream s;
    (s << ... << parts);
    return s.str();
}

// A status other than 0; Fp8qError where it reaches Python through this module
struct StatusError : std::runtime_error {
    fp8q_status status;
    const char* call;
    StatusError(fp8q_status st, const char* what)
        : std::runtime_error(text(what, ": ", fp8q_status_string(st))), status(st), call(what) {}
};
void check(fp8q_status st, const char* what) {
    if (st != FP8Q_OK) throw StatusError(st, what);
}

fp8q_dtype dtype_code(const Tensor& t, const char* name) {
    switch (t.scalar_type()) {
        case at::kFloat: return FP8Q_F32;
        case at::kHalf: return FP8Q_F16;
        case at::kBFloat16: return FP8Q_BF16;
        default: throw py::type_error(text(name, ": only float32, float16 and bfloat16 are allowed, got ", t.scalar_type()));
    }
}

bool is_byte(const Tensor& t) {
    return t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kFloat8_e5m2;
}

void need(const Tensor& t, int64_t numel, const char* name) {
    if (t.numel() < numel) throw py::value_error(text(name, " holds ", t.numel(), " elements, needs ", numel));
}
void need(const Tensor& t, int64_t numel, const char* name, at::ScalarType dtype) {
    if (t.scalar_type() != dtype) throw py::type_error(text(name, " must be ", dtype, ", got ", t.scalar_type()));
    need(t, numel, name);
}
void need_bytes(const Tensor& t, int64_t numel, const char* name) {
    if (!is_byte(t)) throw py::type_error(text(name, " must be uint8 or a float8 dtype, got ", t.scalar_type()));
    need(t, numel, name);
}

// Device pointer of a contiguous CUDA tensor (null for an empty or absent one)
void* pointer(const Tensor& t, const char* name, const Tensor* like = nullptr) {
    if (!t.defined()) return nullptr;
    if (!t.is_cuda()) throw py::value_error(text(name, " must be a CUDA tensor (libfp8q takes device pointers)"));
    if (like && t.device() != like->device())
        throw py::value_error(text(name, " is on ", t.device(), ", expected ", like->device()));
    if (!t.is_contiguous()) throw py::value_error(text(name, " must be contiguous"));
    return t.numel() > 0 ? t.data_ptr() : nullptr;
}
void* pointer(const MaybeTensor& t, const char* name, const Tensor& like) {
    return t ? pointer(*t, name, &like) : nullptr;
}
template <typename T>
T* pointer_as(const Tensor& t, const char* name, const Tensor* like = nullptr) {
    return static_cast<T*>(pointer(t, name, like));
}

// The library sizes its launches from the current device, so a tensor on another one is refused.
fp8q_stream_t stream_of(const Tensor& t, const std::optional<int64_t>& given = std::nullopt) {
    const int current = c10::cuda::current_device();
    if (t.device().index() != current)
        throw py::value_error(text("tensors are on ", t.device(), " but the current device is cuda:", current,
                                   "; call under torch.cuda.device(", static_cast<int>(t.device().index()), ")"));
    if (given) return reinterpret_cast<fp8q_stream_t>(*given);
    return reinterpret_cast<fp8q_stream_t>(at::cuda::getCurrentCUDAStream(t.device().index()).stream());
}

// The stream of a call on x's device, which every other tensor given must be on
template <typename... Others>
fp8q_stream_t on_device(const Tensor& x, const Others&... others) {
    if (!x.is_cuda()) throw py::value_error("the input must be a CUDA tensor (libfp8q takes device pointers)");
    auto same = [&](const Tensor& t) {
        if (t.defined() && t.device() != x.device())
            throw py::value_error(text("a tensor is on ", t.device(), ", expected ", x.device()));
    };
    (same(others), ...);
    return stream_of(x);
}

// memory on x's device, from the caching allocator without a turn through the dispatcher
Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype, const Tensor& x) {
    return Tensor(at::detail::empty_cuda(sizes, dtype, x.device(), std::nullopt));
}

std::string shape_of(const Tensor& t) {
    return text(t.sizes());
}

// rows and width of x[..., n] normed over its last dimension by weight[n]
std::pair<int64_t, int64_t> rows_of(const Tensor& x, const Tensor& weight) {
    if (x.dim() < 1 || weight.dim() != 1 || x.size(-1) != weight.size(0))
        throw py::value_error(text("x must be [..., n] and weight [n], got ", shape_of(x), " and ", shape_of(weight)));
    const int64_t n = weight.size(0);
    return {n ? x.numel() / n : 0, n};
}

void like(const MaybeTensor& t, const Tensor& x, const char* name) {
    if (t && (t->sizes() != x.sizes() || t->scalar_type() != x.scalar_type()))
        throw py::value_error(text(name, " must have x's shape and dtype, got ", shape_of(*t), " ", t->scalar_type()));
}

// The gradients of a function that can be differentiated once: under create_graph they carry a
// node that raises when it is differentiated.
variable_list once(variable_list grads, bool graph, const char* name) {
    if (!graph) return grads;
    for (Tensor& g : grads) {
        if (!g.defined()) continue;
        torch::autograd::DelayedError error(text("trying to differentiate ", name, " twice, which is not supported"), 1);
        Tensor leaf = g.detach();
        leaf.set_requires_grad(true);
        g = error({leaf})[0];
    }
    return grads;
}

// ---------------------------------------------------------------------------
// root-mean-square norm
// ---------------------------------------------------------------------------
void rms_norm_quant(const Tensor& x, const Tensor& weight, const MaybeTensor& y, const MaybeTensor& q,
                    const MaybeTensor& scale_inv, const MaybeTensor& residual, const MaybeTensor& residual_out,
                    const MaybeTensor& rstd, double eps, int64_t group, int fmt, int rule,
                    const std::optional<int64_t>& stream) {
    const auto [m, n] = rows_of(x, weight);
    like(residual, x, "residual");
    like(residual_out, x, "residual_out");
    if (residual.has_value() != residual_out.has_value()) throw py::value_error("residual and residual_out go together");
    if (!y && !q) throw py::value_error("y or q must be given");
    if (y) need(*y, m * n, "y", x.scalar_type());
    if (q) {
        need_bytes(*q, m * n, "q");
        if (!scale_inv) throw py::value_error("q needs scale_inv");
        if (group > 0 && n % group == 0) need(*scale_inv, m * (n / group), "scale_inv", at::kFloat);
    }
    if (rstd) need(*rstd, m, "rstd", at::kFloat);
    void* px = pointer(x, "x");
    const fp8q_dtype xt = dtype_code(x, "x"), wt = dtype_code(weight, "weight");
    void* pr = pointer(residual, "residual", x);
    void* po = pointer(residual_out, "residual_out", x);
    void* pw = pointer(weight, "weight", &x);
    void* py_ = pointer(y, "y", x);
    auto* pq = static_cast<uint8_t*>(pointer(q, "q", x));
    auto* ps = static_cast<float*>(pointer(scale_inv, "scale_inv", x));
    auto* pd = static_cast<float*>(pointer(rstd, "rstd", x));
    if (group < INT_MIN || group > INT_MAX) group = 0;          // refused by the library
    check(fp8q_rms_norm_quant(px, xt, pr, po, pw, wt, m, n, static_cast<float>(eps), static_cast<int>(group),
                              static_cast<fp8q_format>(fmt), static_cast<fp8q_scale_rule>(rule), py_, pq, ps, pd,
                              stream_of(x, stream)),
          "fp8q_rms_norm_quant");
}

// rms_norm and its gradient; keeps the summed rows, the weight and one rstd per row
struct RmsNorm : torch::autograd::Function<RmsNorm> {
    static variable_list forward(AutogradContext* ctx, const Tensor& x_in, const Tensor& weight_in,
                                 const MaybeTensor& residual_in, double eps) {
        const fp8q_stream_t st = on_device(x_in, weight_in, residual_in ? *residual_in : Tensor());
        like(residual_in, x_in, "residual");
        const Tensor x = x_in.contiguous(), weight = weight_in.contiguous();
        const auto [m, n] = rows_of(x, weight);
        const fp8q_dtype xt = dtype_code(x, "x"), wt = dtype_code(weight, "weight");
        Tensor y = empty(x.sizes(), x.scalar_type(), x), rstd = empty({m}, at::kFloat, x), residual, r;
        if (residual_in) {
            residual = residual_in->contiguous();
            r = empty(x.sizes(), x.scalar_type(), x);
        }
        check(fp8q_rms_norm_quant(x.data_ptr(), xt, r.defined() ? residual.data_ptr() : nullptr,
                                  r.defined() ? r.data_ptr() : nullptr, weight.data_ptr(), wt, m, n,
                                  static_cast<float>(eps), 1, FP8Q_E4M3FN, FP8Q_SCALE_IEEE, y.data_ptr(), nullptr, nullptr,
                                  rstd.data_ptr<float>(), st),
              "fp8q_rms_norm_quant");
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({r.defined() ? r : x, weight, rstd});
        return r.defined() ? variable_list{y, r} : variable_list{y};
    }

    static variable_list backward(AutogradContext* ctx, variable_list grads) {
        const bool graph = at::GradMode::is_enabled(), has_residual = grads.size() == 2;
        at::AutoGradMode off(false);
        const Tensor dr_in = has_residual ? grads[1] : Tensor();
        if (!grads[0].defined())                    // only the sum was used: its gradient as it is
            return {dr_in, Tensor(), dr_in, Tensor()};
        const variable_list saved = ctx->get_saved_variables();
        const Tensor &r = saved[0], &weight = saved[1], &rstd = saved[2];
        const fp8q_stream_t st = on_device(r, grads[0], dr_in);
        const Tensor dy = grads[0].contiguous(), dr = dr_in.defined() ? dr_in.contiguous() : Tensor();
        const auto [m, n] = rows_of(r, weight);
        Tensor dx = empty(r.sizes(), r.scalar_type(), r), dw, workspace;
        size_t bytes = 0;
        if (ctx->needs_input_grad(1)) {
            dw = empty(weight.sizes(), weight.scalar_type(), r);
            // a workspace of this call's own: the caching allocator orders it by stream and by graph
            bytes = fp8q_rms_norm_bwd_workspace_bytes(m, n);
            if (bytes) workspace = empty({static_cast<int64_t>(bytes)}, at::kByte, r);
        }
        check(fp8q_rms_norm_bwd(dy.data_ptr(), r.data_ptr(), dtype_code(r, "x"), weight.data_ptr(),
                                dtype_code(weight, "weight"), rstd.data_ptr<float>(), dr.defined() ? dr.data_ptr() : nullptr,
                                m, n, dx.data_ptr(), dw.defined() ? dw.data_ptr() : nullptr,
                                bytes ? workspace.data_ptr() : nullptr, bytes, st),
              "fp8q_rms_norm_bwd");
        return once({dx, dw, has_residual ? dx : Tensor(), Tensor()}, graph, "rms_norm");
    }
};

py::object rms_norm(const Tensor& x, const Tensor& weight, const MaybeTensor& residual, double eps) {
    variable_list out;
    {
        py::gil_scoped_release release;
        out = RmsNorm::apply(x, weight, residual, eps);
    }
    if (!residual) return py::cast(out[0]);
    return py::make_tuple(out[0], out[1]);
}

// ---------------------------------------------------------------------------
// gated feed-forward block
// ---------------------------------------------------------------------------
// an unknown number is refused by the library, not cut to one that there is
fp8q_activation activation(int64_t act) {
    return static_cast<fp8q_activation>(act < 0 || act > INT_MAX ? -1 : act);
}

struct Operands {
    int64_t M, I, K;
    fp8q_format fa, fb;
};
fp8q_format format_of(const Tensor& t, const std::optional<int>& given) {
    if (given) return static_cast<fp8q_format>(*given);
    return t.scalar_type() == at::kFloat8_e5m2 ? FP8Q_E5M2 : FP8Q_E4M3FN;
}
Operands operands(const Tensor& a, const Tensor& w_gate, const Tensor& w_up, const std::optional<int>& fa,
                  const std::optional<int>& fb) {
    if (a.dim() != 2 || w_gate.dim() != 2 || w_up.sizes() != w_gate.sizes() || a.size(1) != w_gate.size(1))
        throw py::value_error(text("a must be [M, K], w_gate and w_up [I, K], got ", shape_of(a), ", ", shape_of(w_gate),
                                   " and ", shape_of(w_up)));
    if (w_gate.scalar_type() != w_up.scalar_type()) throw py::type_error("w_gate and w_up must have one dtype");
    need_bytes(a, 0, "a");
    need_bytes(w_gate, 0, "w_gate");
    return {a.size(0), w_gate.size(0), a.size(1), format_of(a, fa), format_of(w_gate, fb)};
}

uint32_t* status_word(const MaybeTensor& status, const Tensor& a) {
    if (!status) return nullptr;
    if ((status->scalar_type() != at::kInt && status->scalar_type() != at::kUInt32) || status->numel() < 1)
        throw py::type_error("status must be a CUDA int32 or uint32 tensor of at least one element");
    return static_cast<uint32_t*>(pointer(*status, "status", &a));
}

int64_t fine_scales(const Operands& o, const Tensor& scale_a, const Tensor& scale_gate, const Tensor& scale_up) {
    const int64_t kb = (o.K + 127) / 128, ib = (o.I + 127) / 128;
    need(scale_a, o.M * kb, "scale_a", at::kFloat);
    need(scale_gate, ib * kb, "scale_gate", at::kFloat);
    need(scale_up, ib * kb, "scale_up", at::kFloat);
    return ib;
}

void gated_mm_blockwise(const Tensor& a, const Tensor& scale_a, const Tensor& w_gate, const Tensor& scale_gate,
                        const Tensor& w_up, const Tensor& scale_up, const Tensor& out, int act,
                        const std::optional<int>& fa, const std::optional<int>& fb, const MaybeTensor& status,
                        const std::optional<int64_t>& stream) {
    const Operands o = operands(a, w_gate, w_up, fa, fb);
    fine_scales(o, scale_a, scale_gate, scale_up);
    need(out, o.M * o.I, "out");
    auto* pa = pointer_as<uint8_t>(a, "a");
    check(fp8q_gated_mm_blockwise(
              pa, o.fa, pointer_as<float>(scale_a, "scale_a", &a), pointer_as<uint8_t>(w_gate, "w_gate", &a),
              pointer_as<float>(scale_gate, "scale_gate", &a), pointer_as<uint8_t>(w_up, "w_up", &a),
              pointer_as<float>(scale_up, "scale_up", &a), o.fb, o.M, o.I, o.K, activation(act),
              dtype_code(out, "out"), pointer(out, "out", &a), status_word(status, a), stream_of(a, stream)),
          "fp8q_gated_mm_blockwise");
}

void gated_mm_blockwise_quant(const Tensor& a, const Tensor& scale_a, const Tensor& w_gate, const Tensor& scale_gate,
                              const Tensor& w_up, const Tensor& scale_up, const Tensor& q, const Tensor& scale_inv, int act,
                              const std::optional<int>& fa, const std::optional<int>& fb, int fmt, int rule,
                              const MaybeTensor& status, const std::optional<int64_t>& stream) {
    const Operands o = operands(a, w_gate, w_up, fa, fb);
    const int64_t ib = fine_scales(o, scale_a, scale_gate, scale_up);
    need_bytes(q, o.M * o.I, "q");
    need(scale_inv, o.M * ib, "scale_inv", at::kFloat);
    auto* pa = pointer_as<uint8_t>(a, "a");
    check(fp8q_gated_mm_blockwise_quant(
              pa, o.fa, pointer_as<float>(scale_a, "scale_a", &a), pointer_as<uint8_t>(w_gate, "w_gate", &a),
              pointer_as<float>(scale_gate, "scale_gate", &a), pointer_as<uint8_t>(w_up, "w_up", &a),
              pointer_as<float>(scale_up, "scale_up", &a), o.fb, o.M, o.I, o.K, activation(act),
              static_cast<fp8q_format>(fmt), static_cast<fp8q_scale_rule>(rule), pointer_as<uint8_t>(q, "q", &a),
              pointer_as<float>(scale_inv, "scale_inv", &a), status_word(status, a), stream_of(a, stream)),
          "fp8q_gated_mm_blockwise_quant");
}

int64_t rows_before_last(at::IntArrayRef shape) {
    int64_t rows = 1;
    for (size_t i = 0; i + 1 < shape.size(); ++i) rows *= shape[i];
    return rows;
}

// Parts of one buffer, each at a multiple of 256 bytes
template <size_t N>
struct Parts {
    std::array<int64_t, N> at;
    int64_t bytes = 0;
    explicit Parts(const std::array<int64_t, N>& sizes) {
        for (size_t i = 0; i < N; ++i) {
            at[i] = bytes;
            bytes += (sizes[i] + 255) & ~int64_t{255};
        }
    }
};

// gated_linear_fp8: linear_fp8's per-tensor casts and products around the gated kernel and its
// gradient.  Keeps one buffer for the backward pass: the input's and the weight's codes and scales,
// and gate and up in the input's dtype.  Workspaces are the call's own, so that streams and graphs
// share none.
struct GatedLinear : torch::autograd::Function<GatedLinear> {
    static size_t cast_workspace() {
        static const size_t bytes = fp8q_cast_per_tensor_workspace_bytes();
        return bytes;
    }
    // x8, w8, sx, sw, workspace, gate_up
    static Parts<6> parts(int64_t T, int64_t I, int64_t K, int64_t element, bool keep) {
        return Parts<6>({T * K, 2 * I * K, 4, 4, static_cast<int64_t>(cast_workspace()), keep ? 2 * T * I * element : 0});
    }

    static variable_list forward(AutogradContext* ctx, const Tensor& x_in, const Tensor& w_in, int64_t act_in, bool keep) {
        const fp8q_activation act = activation(act_in);
        if ((x_in.scalar_type() != at::kBFloat16 && x_in.scalar_type() != at::kHalf) || x_in.scalar_type() != w_in.scalar_type())
            throw py::type_error("Only float16 and bfloat16 are allowed.");
        if (x_in.dim() < 1 || w_in.dim() != 2 || w_in.size(0) % 16 || x_in.size(-1) != w_in.size(1) || w_in.size(1) % 16)
            throw py::value_error(text("weight must be [2 I, K] with 2 I and K multiples of 16 and K the input's width, got ",
                                       shape_of(w_in), " for an input of ", shape_of(x_in)));
        const fp8q_stream_t st = on_device(x_in, w_in);
        const fp8q_dtype dt = dtype_code(x_in, "input");
        const Tensor x = x_in.contiguous(), w = w_in.contiguous();
        const int64_t I = w.size(0) / 2, K = w.size(1), T = rows_before_last(x.sizes());
        std::vector<int64_t> shape = x.sizes().vec();
        shape.back() = I;
        Tensor h = empty(shape, x.scalar_type(), x);
        const Parts<6> at_ = parts(T, I, K, x.element_size(), keep);
        const Tensor buf = empty({at_.bytes}, at::kByte, x);
        uint8_t* b = static_cast<uint8_t*>(buf.data_ptr());
        uint8_t *x8 = b + at_.at[0], *w8 = b + at_.at[1];
        auto *sx = reinterpret_cast<float*>(b + at_.at[2]), *sw = reinterpret_cast<float*>(b + at_.at[3]);
        check(fp8q_cast_per_tensor_pair(x.data_ptr(), T * K, x8, sx, w.data_ptr(), 2 * I * K, w8, sw, dt, FP8Q_E4M3FN,
                                        b + at_.at[4], cast_workspace(), FP8Q_SCALE_IEEE, st),
              "fp8q_cast_per_tensor_pair");
        check(fp8q_gated_mm(x8, FP8Q_E4M3FN, w8, w8 + I * K, FP8Q_E4M3FN, T, I, K, sx, sw, sw,
                            act, dt, h.data_ptr(), keep ? b + at_.at[5] : nullptr, nullptr, st),
              "fp8q_gated_mm");
        if (keep) {
            ctx->save_for_backward({buf});
            ctx->saved_data["k_act"] = 2 * K + act;           // the other sizes are the gradient's
        }
        return {h};
    }

    static variable_list backward(AutogradContext* ctx, variable_list grads) {
        const bool graph = at::GradMode::is_enabled();
        at::AutoGradMode off(false);
        const Tensor buf = ctx->get_saved_variables()[0];
        const fp8q_stream_t st = on_device(buf, grads[0]);
        const Tensor dh = grads[0].contiguous();
        const int64_t k_act = ctx->saved_data["k_act"].toInt(), K = k_act / 2;
        const auto act = static_cast<fp8q_activation>(k_act % 2);
        const int64_t I = dh.size(-1), T = rows_before_last(dh.sizes());
        const Parts<6> at_ = parts(T, I, K, dh.element_size(), true);
        uint8_t* b = static_cast<uint8_t*>(buf.data_ptr());
        const uint8_t *x8 = b + at_.at[0], *w8 = b + at_.at[1];
        const auto *sx = reinterpret_cast<const float*>(b + at_.at[2]), *sw = reinterpret_cast<const float*>(b + at_.at[3]);
        const fp8q_dtype dt = dtype_code(dh, "the gradient");
        const Parts<3> to({2 * T * I, 4, static_cast<int64_t>(cast_workspace())});
        const Tensor tmp = empty({to.bytes}, at::kByte, buf);
        uint8_t* d8 = static_cast<uint8_t*>(tmp.data_ptr());
        float* sd = reinterpret_cast<float*>(d8 + to.at[1]);
        check(fp8q_gated_bwd_cast(dh.data_ptr(), b + at_.at[5], dt, T, I, act, FP8Q_E5M2, d8, sd, d8 + to.at[2],
                                  cast_workspace(), FP8Q_SCALE_IEEE, st),
              "fp8q_gated_bwd_cast");
        Tensor dx, dw;
        if (ctx->needs_input_grad(0)) {
            // dx[T, K] = d[T, 2 I] @ w[2 I, K], one product over gate's and up's columns together
            std::vector<int64_t> shape = dh.sizes().vec();
            shape.back() = K;
            dx = empty(shape, dh.scalar_type(), buf);
            check(fp8q_scaled_mm_ex(d8, FP8Q_E5M2, FP8Q_K_MAJOR, w8, FP8Q_E4M3FN, FP8Q_MN_MAJOR, T, K, 2 * I, sd, sw, nullptr,
                                    dt, dx.data_ptr(), nullptr, st),
                  "fp8q_scaled_mm_ex");
        }
        if (ctx->needs_input_grad(1)) {
            // dw[2 I, K] = d^T[2 I, T] @ x[T, K], any token count
            dw = empty({2 * I, K}, dh.scalar_type(), buf);
            check(fp8q_scaled_mm_ex(d8, FP8Q_E5M2, FP8Q_MN_MAJOR, x8, FP8Q_E4M3FN, FP8Q_MN_MAJOR, 2 * I, K, T, sd, sx, nullptr,
                                    dt, dw.data_ptr(), nullptr, st),
                  "fp8q_scaled_mm_ex");
        }
        return once({dx, dw, Tensor(), Tensor()}, graph, "gated_linear_fp8");
    }
};

Tensor gated_linear_fp8(const Tensor& x, const Tensor& w, int64_t act) {
    const bool keep = at::GradMode::is_enabled() && (x.requires_grad() || w.requires_grad());
    return GatedLinear::apply(x, w, act, keep)[0];
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
    m.doc() = "The norm and feed-forward calls of libfp8q: marshalling and autograd";
    m.attr("built_for") = FP8Q_BUILT_FOR;          // the build looks for it in the file
    py::register_local_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const StatusError& e) {
            py::object error = py::module_::import("dequantisation_fp8q_token_b200").attr("Fp8qError");
            PyErr_SetObject(error.ptr(), error(static_cast<int>(e.status), e.call).ptr());
        }
    });
    // a launch may wait for the device: never with the interpreter locked
    using Unlocked = py::call_guard<py::gil_scoped_release>;
    m.def("rms_norm_quant", &rms_norm_quant, Unlocked());
    m.def("rms_norm", &rms_norm);
    m.def("gated_mm_blockwise", &gated_mm_blockwise, Unlocked());
    m.def("gated_mm_blockwise_quant", &gated_mm_blockwise_quant, Unlocked());
    m.def("gated_linear_fp8", &gated_linear_fp8, Unlocked());
}
