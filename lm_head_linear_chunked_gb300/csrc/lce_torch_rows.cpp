// The torch side of the operators between token ids and the head (RMS norm,
// embedding, rows sorted by expert), in compiled code like lce_torch.cpp's and
// for its reason: their small calls are bound by the host.
#include "lce_torch.h"

using namespace lce_torch;

namespace {

// The sizes of all dimensions but the last, and a last one of n.
std::vector<int64_t> with_last(at::IntArrayRef sizes, int64_t n) {
    std::vector<int64_t> v = sizes.vec();
    v.back() = n;
    return v;
}
std::vector<int64_t> and_last(at::IntArrayRef sizes, int64_t n) {
    std::vector<int64_t> v = sizes.vec();
    v.push_back(n);
    return v;
}

int index_bytes(const Tensor& t, const char* what) {
    if (t.scalar_type() == at::kLong) return 8;
    if (t.scalar_type() == at::kInt) return 4;
    throw py::type_error(std::string(what) + " must be int32 or int64, got " + toString(t.scalar_type()));
}

// ---------------------------------------------------------------- RMS norm

struct RmsIn {
    int code, wcode;
    int64_t rows, H, ldx = 0, ldr = 0;
    Tensor x;
    OptTensor residual, weight;
};

RmsIn rms_in(const Tensor& x, const OptTensor& weight, const OptTensor& residual) {
    no_tangent(x, "x");
    no_tangent(weight, "weight");
    no_tangent(residual, "residual");
    RmsIn in;
    in.code = in.wcode = type_code(x, "x");
    in.H = width(x);
    if (weight) {
        check_affine(x, in.H, *weight, "weight");
        in.wcode = type_code(*weight, "weight");
    }
    if (residual) {
        check_shape(*residual, x.sizes(), "residual");
        check_type(*residual, x.scalar_type(), "residual");
    }
    const at::Device dev = x.device();
    on_cuda(dev);
    on_device(weight, dev, "weight");
    on_device(residual, dev, "residual");
    in.rows = x.numel() / in.H;
    return in;
}

Tensor plain(const Tensor& t) { return t.is_neg() ? t.resolve_neg().contiguous() : t.contiguous(); }

// The rows, on their device (under the caller's guard).
void rms_rows(RmsIn* in, const Tensor& x, const OptTensor& weight, const OptTensor& residual) {
    in->x = rows_of(x, &in->ldx);
    in->ldr = in->ldx;
    if (residual) in->residual = rows_of(*residual, &in->ldr);
    if (weight) in->weight = plain(*weight);
}

// y, and where wanted the sum and rstd
std::tuple<Tensor, OptTensor, OptTensor> rms_forward(const Tensor& x, const OptTensor& weight, const OptTensor& residual,
                                                     double eps, bool stats, bool recorded) {
    if (!recorded) not_traced("rms_norm_forward");
    RmsIn in = rms_in(x, weight, residual);
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    rms_rows(&in, x, weight, residual);
    const Tensor y = like(in.x);
    OptTensor sum, rstd;
    if (residual) sum = like(in.x);
    if (stats) rstd = empty({in.rows}, at::kFloat, dev);
    check(lib.rms_forward(in.rows, in.H, in.code, in.wcode, in.x.data_ptr(), in.ldx, ptr(in.residual), in.ldr, ptr(in.weight),
                          static_cast<float>(eps), ptr(sum), in.H, y.data_ptr(), in.H, static_cast<float*>(ptr(rstd)),
                          stream_of(dev)),
          "lce_rms_norm_forward");
    return {y, sum, rstd};
}

// q, the scales and, with a residual, the sum
std::tuple<Tensor, Tensor, OptTensor> rms_fp8(const Tensor& x, const OptTensor& weight, const OptTensor& residual, double eps,
                                              int64_t group) {
    not_traced("rms_norm_fp8");
    if (group != 0 && group != LCE_FP8_GROUP)
        throw py::value_error("group must be 0 (the row) or " + std::to_string(LCE_FP8_GROUP) + ", got " + std::to_string(group));
    RmsIn in = rms_in(x, weight, residual);
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    rms_rows(&in, x, weight, residual);
    const Tensor q = empty(x.sizes(), at::kFloat8_e4m3fn, dev);
    const Tensor scales = empty(with_last(x.sizes(), group ? (in.H + group - 1) / group : 1), at::kFloat, dev);
    OptTensor sum;
    if (residual) sum = like(in.x);
    check(lib.rms_fp8(in.rows, in.H, in.code, in.wcode, in.x.data_ptr(), in.ldx, ptr(in.residual), in.ldr, ptr(in.weight),
                      static_cast<float>(eps), ptr(sum), in.H, static_cast<uint8_t*>(q.data_ptr()), in.H, ptr<float>(scales),
                      group, stream_of(dev)),
          "lce_rms_norm_fp8");
    return {q, scales, sum};
}

std::tuple<OptTensor, OptTensor> rms_backward(const Tensor& dy_in, const Tensor& x_in, const OptTensor& weight,
                                              const Tensor& rstd, const OptTensor& ds_in, bool want_x, bool want_w) {
    not_traced("rms_norm_backward");
    no_tangent(dy_in, "grad_y");
    no_tangent(x_in, "x");
    no_tangent(weight, "weight");
    no_tangent(rstd, "rstd");
    no_tangent(ds_in, "grad_sum");
    const int code = type_code(x_in, "x");
    const int64_t H = width(x_in), rows = x_in.numel() / H;
    check_shape(dy_in, x_in.sizes(), "grad_y");
    check_type(dy_in, x_in.scalar_type(), "grad_y");
    if (weight) check_affine(x_in, H, *weight, "weight");
    want_w = want_w && weight.has_value();
    check_shape(rstd, {rows}, "rstd");
    check_type(rstd, at::kFloat, "rstd");
    if (!rstd.is_contiguous() || rstd.is_neg()) throw py::type_error("rstd must be contiguous");
    if (ds_in) {
        check_shape(*ds_in, x_in.sizes(), "grad_sum");
        check_type(*ds_in, x_in.scalar_type(), "grad_sum");
    }
    const at::Device dev = x_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(dy_in, dev, "grad_y");
    on_device(weight, dev, "weight");
    on_device(rstd, dev, "rstd");
    on_device(ds_in, dev, "grad_sum");
    int64_t ldx = 0, ldd = 0, ldds = 0;
    const Tensor x = rows_of(x_in, &ldx), dy = rows_of(dy_in, &ldd);
    OptTensor ds, dx, dw, ws, w;
    if (weight) w = plain(*weight);
    if (ds_in) ds = rows_of(*ds_in, &ldds);
    if (want_x) dx = like(x);
    size_t bytes = 0;
    if (want_w) {
        dw = empty({H}, weight->scalar_type(), dev);
        check(lib.rms_workspace(rows, H, &bytes), "lce_rms_norm_workspace_size");
        ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
    }
    if (want_x || want_w)
        check(lib.rms_backward(rows, H, code, weight ? type_code(*weight, "weight") : code, dy.data_ptr(), ldd, x.data_ptr(), ldx,
                               ptr(w), ptr<float>(rstd), ptr(ds), ldds, ptr(dx), H, ptr(dw), ptr(ws), bytes,
                               stream_of(dev)),
              "lce_rms_norm_backward");
    return {dx, dw};
}

// ---------------------------------------------------------------- embedding

void check_matrix(const Tensor& t, const char* what) {
    if (t.dim() != 2 || t.size(1) == 0) throw py::value_error(std::string(what) + " must be a matrix, got " + text(t.sizes()));
}

Tensor embedding_forward(const Tensor& tokens_in, const Tensor& weight, double scale, std::optional<int64_t> padding,
                         const OptTensor& status, bool recorded) {
    if (!recorded) not_traced("embedding_forward");
    no_tangent(weight, "weight");
    const int code = type_code(weight, "weight"), bytes = index_bytes(tokens_in, "tokens");
    check_matrix(weight, "weight");
    const int64_t V = weight.size(0), H = weight.size(1);
    const at::Device dev = weight.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(tokens_in, dev, "tokens");
    int64_t ldw = 0;
    const Tensor w = rows_of(weight, &ldw), tokens = tokens_in.contiguous();
    const Tensor y = empty(and_last(tokens.sizes(), H), weight.scalar_type(), dev);
    check(lib.embedding_forward(tokens.numel(), V, H, code, tokens.data_ptr(), bytes, w.data_ptr(), ldw,
                                static_cast<float>(scale), padding.value_or(LCE_NO_PADDING), y.data_ptr(), H, ptr(status),
                                stream_of(dev)),
          "lce_embedding_forward");
    return y;
}

// out [n, H], rows apart by its stride, must not reach into the memory that `in` may lie in, unless the rows of both are
// other columns of one buffer.
void apart(const Tensor& out, int64_t n, int64_t H, const Tensor& in, const char* what) {
    if (!out.has_storage() || !in.has_storage() || !out.numel() || !in.numel()) return;
    const auto first = reinterpret_cast<uintptr_t>(out.const_data_ptr()), from = reinterpret_cast<uintptr_t>(in.const_data_ptr());
    const int64_t es = static_cast<int64_t>(in.element_size());
    if (n > 1) {
        const int64_t step = out.stride(0) * static_cast<int64_t>(out.element_size());
        int64_t column = static_cast<int64_t>(from - first) % step;
        if (column < 0) column += step;
        bool rows = in.size(-1) == 1 || in.stride(-1) == 1;
        for (int64_t d = 0; d + 1 < in.dim(); ++d) rows &= in.size(d) == 1 || in.stride(d) * es % step == 0;
        if (rows && column >= H * static_cast<int64_t>(out.element_size()) && column + in.size(-1) * es <= step) return;
    }
    int64_t last = 0;
    for (int64_t d = 0; d < in.dim(); ++d) last += (in.size(d) - 1) * in.stride(d);
    const uintptr_t end = first + ((n > 1 ? (n - 1) * out.stride(0) : 0) + H) * out.element_size();
    if (first < from + (last + 1) * es && from < end) throw py::value_error(std::string("out and ") + what + " overlap");
}

// grad_weight and the workspace
std::tuple<Tensor, Tensor> embedding_backward(const Tensor& dy_in, const Tensor& tokens_in, int64_t V, double scale,
                                              std::optional<int64_t> padding, std::optional<at::ScalarType> type,
                                              const OptTensor& out, bool accumulate) {
    not_traced("embedding_backward");
    no_tangent(dy_in, "grad_y");
    no_tangent(out, "out");
    const int code = type_code(dy_in, "grad_y"), bytes = index_bytes(tokens_in, "tokens");
    const int64_t H = width(dy_in);
    check_shape(dy_in, and_last(tokens_in.sizes(), H), "grad_y");
    if (V <= 0) throw py::value_error("the vocabulary must not be empty");
    const at::ScalarType gtype = type.value_or(out ? out->scalar_type() : dy_in.scalar_type());
    if (gtype != dy_in.scalar_type() && gtype != at::kFloat)
        throw py::type_error(std::string("grad_weight must be of grad_y's type or float32, got ") + toString(gtype));
    if (accumulate && !out) throw py::value_error("accumulate needs the running sum as out");
    if (accumulate && gtype != at::kFloat) throw py::type_error(std::string("accumulate needs a float32 sum, got ") + toString(gtype));
    if (out) {
        check_shape(*out, {V, H}, "out");
        check_type(*out, gtype, "out");
        if ((H > 1 && out->stride(1) != 1) || (V > 1 && out->stride(0) < H) || out->is_neg())
            throw py::value_error("out must have contiguous rows that do not overlap, got strides " + text(out->strides()));
        apart(*out, V, H, dy_in, "grad_y");
    }
    const at::Device dev = dy_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(tokens_in, dev, "tokens");
    on_device(out, dev, "out");
    int64_t ldd = 0;
    const Tensor dy = rows_of(dy_in, &ldd), tokens = tokens_in.contiguous();
    const int64_t N = tokens.numel();
    const Tensor dw = out ? *out : empty({V, H}, gtype, dev);
    size_t space = 0;
    check(lib.embedding_workspace(N, V, H, &space), "lce_embedding_workspace_size");
    const Tensor ws = empty({static_cast<int64_t>(space)}, at::kByte, dev);
    check(lib.embedding_backward(N, V, H, code, gtype == at::kFloat ? LCE_F32 : code, tokens.data_ptr(), bytes, dy.data_ptr(), ldd,
                                 static_cast<float>(scale), padding.value_or(LCE_NO_PADDING), dw.data_ptr(),
                                 V > 1 ? dw.stride(0) : H, ws.data_ptr(), space, stream_of(dev), accumulate ? LCE_ACCUMULATE : 0),
          "lce_embedding_backward");
    if (out && !out->is_inference()) out->unsafeGetTensorImpl()->bump_version();  // written, for what has saved it
    return {dw, ws};
}

// ---------------------------------------------------------------- rows sorted by expert

// positions, slots, counts, offsets, ws
std::vector<Tensor> expert_plan(const Tensor& experts_in, int64_t E, const OptTensor& mask_in, int64_t align) {
    not_traced("expert_plan");
    const int bytes = index_bytes(experts_in, "experts");
    if (experts_in.dim() == 0 || experts_in.size(-1) == 0)
        throw py::value_error("experts must have shape [tokens, slots], got " + text(experts_in.sizes()));
    if (mask_in) {
        check_shape(*mask_in, experts_in.sizes().slice(0, experts_in.dim() - 1), "mask");
        check_type(*mask_in, at::kBool, "mask");
    }
    const int64_t k = experts_in.size(-1), T = experts_in.numel() / k;
    int64_t R = 0;
    size_t space = 0;
    check(lib.expert_rows(T, k, E, align, &R), "lce_expert_rows");
    check(lib.expert_plan_workspace(T, k, E, &space), "lce_expert_plan_workspace_size");
    const at::Device dev = experts_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(mask_in, dev, "mask");
    const Tensor experts = experts_in.contiguous();
    OptTensor mask;
    if (mask_in) mask = mask_in->contiguous();
    const auto [positions, slots] = empty_pair(experts.sizes(), {R}, at::kInt, dev);
    const auto [counts, offsets] = empty_pair({E}, {E + 1}, at::kLong, dev);
    std::vector<Tensor> out{positions, slots, counts, offsets, empty({static_cast<int64_t>(space)}, at::kByte, dev)};
    check(lib.expert_plan(T, k, E, align, experts.data_ptr(), bytes, static_cast<const uint8_t*>(ptr(mask)), ptr<int32_t>(out[0]),
                          ptr<int32_t>(out[1]), ptr<int64_t>(out[2]), ptr<int64_t>(out[3]), out[4].data_ptr(), space, stream_of(dev)),
          "lce_expert_plan");
    return out;
}

struct Plan {
    int64_t T, k;
    const int32_t* positions;
    at::IntArrayRef lead;  // the tokens' dimensions
};

Plan plan_of(const Tensor& positions) {
    check_type(positions, at::kInt, "positions");
    if (positions.dim() == 0 || positions.size(-1) == 0 || !positions.is_contiguous())
        throw py::value_error("positions must be a plan's, contiguous and [tokens, slots], got " + text(positions.sizes()));
    const int64_t k = positions.size(-1);
    return {positions.numel() / k, k, ptr<int32_t>(positions), positions.sizes().slice(0, positions.dim() - 1)};
}

void check_slots(const Tensor& slots) {
    check_type(slots, at::kInt, "slots");
    if (slots.dim() != 1 || !slots.is_contiguous()) throw py::value_error("slots must be a plan's, got " + text(slots.sizes()));
}

int64_t token_width(const Plan& plan, const Tensor& t, const char* what) {
    if (t.dim() == 0 || t.size(-1) == 0 || t.sizes().slice(0, t.dim() - 1) != plan.lead)
        throw py::value_error(std::string(what) + " must have shape " + text(plan.lead) + " + [columns], got " + text(t.sizes()));
    return t.size(-1);
}

Tensor expert_dispatch(const Tensor& x_in, const Tensor& positions, const Tensor& slots, bool recorded) {
    if (!recorded) not_traced("dispatch_forward");
    no_tangent(x_in, "x");
    const int code = type_code(x_in, "x");
    const Plan plan = plan_of(positions);
    check_slots(slots);
    const int64_t H = token_width(plan, x_in, "x"), R = slots.size(0);
    const at::Device dev = x_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(positions, dev, "positions");
    on_device(slots, dev, "slots");
    int64_t ldx = 0;
    const Tensor x = rows_of(x_in, &ldx);
    const Tensor rows = empty({R, H}, x.scalar_type(), dev);
    check(lib.expert_dispatch(plan.T, plan.k, H, R, code, x.data_ptr(), ldx, plan.positions, ptr<int32_t>(slots), rows.data_ptr(), H,
                              stream_of(dev)),
          "lce_expert_dispatch");
    return rows;
}

int check_weights(const Tensor& weights, const Tensor& rows, const Tensor& positions) {
    check_shape(weights, positions.sizes(), "weights");
    if (weights.scalar_type() != rows.scalar_type()) check_type(weights, at::kFloat, "weights");
    return type_code(weights, "weights");
}

Tensor expert_combine(const Tensor& rows_in, const OptTensor& weights_in, const Tensor& positions, const Tensor& slots,
                      bool recorded) {
    if (!recorded) not_traced("combine_forward");
    no_tangent(rows_in, "rows");
    no_tangent(weights_in, "weights");
    const int code = type_code(rows_in, "rows");
    const Plan plan = plan_of(positions);
    check_matrix(rows_in, "rows");
    check_slots(slots);
    int wcode = code;
    if (weights_in) wcode = check_weights(*weights_in, rows_in, positions);
    const int64_t R = slots.size(0), H = rows_in.size(1);
    check_shape(rows_in, {R, H}, "rows");
    const at::Device dev = rows_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(positions, dev, "positions");
    on_device(weights_in, dev, "weights");
    int64_t ldr = 0;
    const Tensor rows = rows_of(rows_in, &ldr);
    OptTensor weights;
    if (weights_in) weights = plain(*weights_in);
    const Tensor y = empty(and_last(plan.lead, H), rows.scalar_type(), dev);
    check(lib.expert_combine(plan.T, plan.k, H, R, code, wcode, rows.data_ptr(), ldr, ptr(weights), plan.positions, y.data_ptr(), H,
                             stream_of(dev)),
          "lce_expert_combine");
    return y;
}

std::tuple<OptTensor, OptTensor> expert_combine_backward(const Tensor& dy_in, const Tensor& rows_in, const OptTensor& weights_in,
                                                         const Tensor& positions, const Tensor& slots, bool want_rows,
                                                         bool want_weights) {
    not_traced("combine_backward");
    no_tangent(dy_in, "grad_y");
    no_tangent(rows_in, "rows");
    no_tangent(weights_in, "weights");
    const int code = type_code(rows_in, "rows");
    const Plan plan = plan_of(positions);
    check_slots(slots);
    check_matrix(rows_in, "rows");
    check_type(dy_in, rows_in.scalar_type(), "grad_y");
    int wcode = code;
    if (weights_in) wcode = check_weights(*weights_in, rows_in, positions);
    want_weights = want_weights && weights_in.has_value();
    const int64_t R = slots.size(0), H = token_width(plan, dy_in, "grad_y");
    check_shape(rows_in, {R, H}, "rows");
    const at::Device dev = rows_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(dy_in, dev, "grad_y");
    on_device(positions, dev, "positions");
    on_device(slots, dev, "slots");
    on_device(weights_in, dev, "weights");
    int64_t ldr = 0, ldd = 0;
    const Tensor rows = rows_of(rows_in, &ldr), dy = rows_of(dy_in, &ldd);
    OptTensor weights, grad_rows, grad_weights;
    if (weights_in) weights = plain(*weights_in);
    if (want_rows) grad_rows = empty({R, H}, rows.scalar_type(), dev);
    if (want_weights) grad_weights = empty(positions.sizes(), weights->scalar_type(), dev);
    check(lib.expert_combine_backward(plan.T, plan.k, H, R, code, wcode, dy.data_ptr(), ldd, rows.data_ptr(), ldr, ptr(weights),
                                      plan.positions, ptr<int32_t>(slots), ptr(grad_rows), H, ptr(grad_weights), stream_of(dev)),
          "lce_expert_combine_backward");
    return {grad_rows, grad_weights};
}

Tensor expert_dispatch_backward(const Tensor& grad_in, const Tensor& positions, const Tensor& slots) {
    not_traced("dispatch_backward");
    no_tangent(grad_in, "grad_rows");
    const int code = type_code(grad_in, "grad_rows");
    const Plan plan = plan_of(positions);
    check_matrix(grad_in, "grad_rows");
    check_slots(slots);
    check_shape(grad_in, {slots.size(0), grad_in.size(1)}, "grad_rows");
    const at::Device dev = grad_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(positions, dev, "positions");
    int64_t ldr = 0;
    const Tensor grad = rows_of(grad_in, &ldr);
    const int64_t R = grad.size(0), H = grad.size(1);
    const Tensor dx = empty(and_last(plan.lead, H), grad.scalar_type(), dev);
    check(lib.expert_dispatch_backward(plan.T, plan.k, H, R, code, grad.data_ptr(), ldr, plan.positions, dx.data_ptr(), H,
                                       stream_of(dev)),
          "lce_expert_dispatch_backward");
    return dx;
}

}  // namespace

void lce_torch::bind_rows(py::module_& m) {
    m.def("rms_forward", &rms_forward);
    m.def("rms_fp8", &rms_fp8);
    m.def("rms_backward", &rms_backward);
    m.def("embedding_forward", &embedding_forward);
    m.def("embedding_backward", &embedding_backward);
    m.def("expert_plan", &expert_plan);
    m.def("expert_dispatch", &expert_dispatch);
    m.def("expert_dispatch_backward", &expert_dispatch_backward);
    m.def("expert_combine", &expert_combine);
    m.def("expert_combine_backward", &expert_combine_backward);
}
