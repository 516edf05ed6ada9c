// The torch side of the operators beside the head: checks of tensors, their
// outputs and workspaces, and one call of the C ABI, in compiled code.  A
// small call is bound by the host (a norm of 16 rows takes 4.9 us, replayed in
// a CUDA graph 2.3; a selection over four beams 10.0 and 7.7), and the same
// steps from Python took two to three times as long (13 and 23 us).  The library
// itself stays behind include/lce.h: its addresses come from the ctypes binding,
// so that both use one library.  What several operators share is in lce_torch.h,
// the operators between token ids and the head are in lce_torch_rows.cpp.
//
// Everything that a kernel would otherwise read through a wrong pointer,
// stride or type is refused here (TypeError, ValueError); a status other than
// LCE_OK raises the package's LCEError.
#include <algorithm>

#include "lce_torch.h"

namespace lce_torch {
Library lib;
PyObject *lce_error = nullptr, *traced_error = nullptr;
}  // namespace lce_torch

using namespace lce_torch;

namespace {

void init(const py::dict& at, const py::object& error, const py::object& traced) {
    auto get = [&](const char* name, auto& f) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>(at[name].cast<uintptr_t>());
    };
    get("lce_layer_norm_forward", lib.norm_forward);
    get("lce_layer_norm_backward", lib.norm_backward);
    get("lce_layer_norm_workspace_size", lib.norm_workspace);
    get("lce_balance_forward", lib.balance_forward);
    get("lce_balance_fused", lib.balance_fused);
    get("lce_balance_backward", lib.balance_backward);
    get("lce_balance_workspace_size", lib.balance_workspace);
    get("lce_beam_select", lib.beam_select);
    get("lce_beam_workspace_size", lib.beam_workspace);
    get("lce_beam_reorder", lib.beam_reorder);
    get("lce_rms_norm_forward", lib.rms_forward);
    get("lce_rms_norm_fp8", lib.rms_fp8);
    get("lce_rms_norm_backward", lib.rms_backward);
    get("lce_rms_norm_workspace_size", lib.rms_workspace);
    get("lce_embedding_forward", lib.embedding_forward);
    get("lce_embedding_backward", lib.embedding_backward);
    get("lce_embedding_workspace_size", lib.embedding_workspace);
    get("lce_expert_rows", lib.expert_rows);
    get("lce_expert_plan", lib.expert_plan);
    get("lce_expert_plan_workspace_size", lib.expert_plan_workspace);
    get("lce_expert_dispatch", lib.expert_dispatch);
    get("lce_expert_dispatch_backward", lib.expert_dispatch_backward);
    get("lce_expert_combine", lib.expert_combine);
    get("lce_expert_combine_backward", lib.expert_combine_backward);
    lce_error = error.inc_ref().ptr();
    traced_error = traced.inc_ref().ptr();
}

// ---------------------------------------------------------------- layer norm

// recorded: called by an autograd function, which a trace records as one call

std::tuple<Tensor, OptTensor, OptTensor> norm_forward(const Tensor& x_in, const OptTensor& weight, const OptTensor& bias,
                                                      double eps, bool stats, bool recorded) {
    if (!recorded) not_traced("layer_norm_forward");
    no_tangent(x_in, "x");
    no_tangent(weight, "weight");
    no_tangent(bias, "bias");
    const int code = type_code(x_in, "x");
    const int64_t H = width(x_in);
    int wcode = code;
    if (weight) {
        check_affine(x_in, H, *weight, "weight");
        wcode = type_code(*weight, "weight");
    }
    if (bias) {
        check_affine(x_in, H, *bias, "bias");
        if (weight) check_type(*bias, weight->scalar_type(), "bias (beside this weight)");
        wcode = type_code(*bias, "bias");
    }
    const at::Device dev = x_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(weight, dev, "weight");
    on_device(bias, dev, "bias");
    int64_t ldx = 0;
    const Tensor x = rows_of(x_in, &ldx);
    const int64_t rows = x.numel() / H;
    const Tensor y = like(x);
    OptTensor mean, rstd;
    if (stats) {
        mean = empty({rows}, at::kFloat, dev);
        rstd = empty({rows}, at::kFloat, dev);
    }
    check(lib.norm_forward(rows, H, code, wcode, x.data_ptr(), ldx, ptr(weight), ptr(bias), static_cast<float>(eps),
                           y.data_ptr(), H, static_cast<float*>(ptr(mean)), static_cast<float*>(ptr(rstd)),
                           stream_of(dev)),
          "lce_layer_norm_forward");
    return {y, mean, rstd};
}

std::tuple<OptTensor, OptTensor, OptTensor> norm_backward(const Tensor& dy_in, const Tensor& x_in, const OptTensor& weight,
                                                          const Tensor& mean, const Tensor& rstd, bool want_x,
                                                          bool want_w, bool want_b,
                                                          std::optional<at::ScalarType> grad_type) {
    not_traced("layer_norm_backward");
    no_tangent(dy_in, "grad_y");
    no_tangent(x_in, "x");
    no_tangent(weight, "weight");
    no_tangent(mean, "mean");
    no_tangent(rstd, "rstd");
    const int code = type_code(x_in, "x");
    const int64_t H = width(x_in);
    check_shape(dy_in, x_in.sizes(), "grad_y");
    check_type(dy_in, x_in.scalar_type(), "grad_y");
    at::ScalarType gtype = grad_type.value_or(x_in.scalar_type());
    if (weight) {
        check_affine(x_in, H, *weight, "weight");
        gtype = weight->scalar_type();
    } else if (gtype != x_in.scalar_type() && gtype != at::kFloat) {
        throw py::type_error(std::string("grad_dtype must be x's or float32, got ") + toString(gtype));
    }
    const int64_t rows = x_in.numel() / H;
    for (const Tensor* t : {&mean, &rstd}) {
        check_shape(*t, {rows}, "mean and rstd");
        check_type(*t, at::kFloat, "mean and rstd");
        if (!t->is_contiguous()) throw py::type_error("mean and rstd must be contiguous");
    }
    const at::Device dev = x_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(dy_in, dev, "grad_y");
    on_device(weight, dev, "weight");
    on_device(mean, dev, "mean");
    on_device(rstd, dev, "rstd");
    int64_t ldx = 0, ldd = 0;
    const Tensor x = rows_of(x_in, &ldx), dy = rows_of(dy_in, &ldd);
    OptTensor dx, dw, db, ws;
    if (want_x) dx = like(x);
    if (want_w) dw = empty({H}, gtype, dev);
    if (want_b) db = empty({H}, gtype, dev);
    size_t bytes = 0;
    if (want_w || want_b) {
        check(lib.norm_workspace(rows, H, &bytes), "lce_layer_norm_workspace_size");
        ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
    }
    if (want_x || want_w || want_b)
        check(lib.norm_backward(rows, H, code, gtype == at::kFloat ? LCE_F32 : code, dy.data_ptr(), ldd, x.data_ptr(),
                                ldx, ptr(weight), ptr<float>(mean), ptr<float>(rstd), ptr(dx), H, ptr(dw), ptr(db),
                                ptr(ws), bytes, stream_of(dev)),
              "lce_layer_norm_backward");
    return {dx, dw, db};
}

// ---------------------------------------------------------------- balance loss

struct Router {
    int64_t G, T, E, zg, zt, mg;
    int code;
    Tensor z;
    OptTensor mask;
};

Router router_of(const Tensor& logits, const OptTensor& mask) {
    no_tangent(logits, "router_logits");
    Router r;
    r.code = type_code(logits, "router_logits");
    const int64_t dim = logits.dim();
    if (dim != 2 && dim != 3)
        throw py::value_error("router_logits must be [tokens, experts] or [groups, tokens, experts], got " + text(logits.sizes()));
    r.T = logits.size(-2);
    r.E = logits.size(-1);
    r.G = dim == 3 ? logits.size(0) : 1;
    if (!r.G || !r.T || !r.E) throw py::value_error("router_logits is empty: " + text(logits.sizes()));
    r.z = logits;
    if (!logits.is_contiguous() && (logits.stride(-1) != 1 || (r.T > 1 && logits.stride(-2) < r.E))) r.z = logits.contiguous();
    r.zg = dim == 3 ? r.z.stride(0) : 0;
    r.zt = r.T > 1 ? r.z.stride(-2) : r.E;
    r.mg = 0;
    if (mask) {
        check_type(*mask, at::kBool, "mask");
        if (mask->dim() == 2 && dim == 3) {
            check_shape(*mask, {r.G, r.T}, "mask");
            r.mg = r.T;
        } else {
            check_shape(*mask, {r.T}, "mask");
        }
        r.mask = mask->contiguous();
    }
    return r;
}

const float* grad_output_of(const OptTensor& t, const at::Device& dev) {
    if (!t) return nullptr;
    if (t->numel() != 1 || t->scalar_type() != at::kFloat) throw py::type_error("grad_output must be one float32 value");
    on_device(*t, dev, "grad_output");
    return ptr<float>(*t);
}

// loss, group_loss, counts, n_valid, ws and (with grad) grad_logits
std::vector<Tensor> balance_call(const Tensor& logits, const Tensor& experts_in, const OptTensor& mask, bool sum, bool grad,
                                 double grad_scale, const OptTensor& grad_output, bool recorded) {
    if (!recorded) not_traced(grad ? "balance_fused" : "balance_forward");
    no_tangent(grad_output, "grad_output");
    const Router r = router_of(logits, mask);
    const int index_bytes = experts_in.scalar_type() == at::kLong ? 8 : experts_in.scalar_type() == at::kInt ? 4 : 0;
    if (!index_bytes) throw py::type_error(std::string("experts must be int32 or int64, got ") + toString(experts_in.scalar_type()));
    const auto lead = logits.sizes().slice(0, logits.dim() - 1);
    if (experts_in.dim() != logits.dim() || experts_in.sizes().slice(0, lead.size()) != lead || experts_in.size(-1) == 0)
        throw py::value_error("experts must have shape " + text(lead) + " + [slots], got " + text(experts_in.sizes()));
    const at::Device dev = logits.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(experts_in, dev, "experts");
    on_device(r.mask, dev, "mask");
    const float* go = grad_output_of(grad_output, dev);
    const Tensor experts = experts_in.contiguous();
    const int64_t k = experts.size(-1);
    size_t bytes = 0;
    check(lib.balance_workspace(r.G, r.T, r.E, k, &bytes), "lce_balance_workspace_size");
    const Tensor loss = empty({1}, at::kFloat, dev), group_loss = empty({r.G}, at::kFloat, dev);
    const Tensor counts = logits.dim() == 3 ? empty({r.G, r.E}, at::kLong, dev) : empty({r.E}, at::kLong, dev);
    const Tensor n_valid = empty({r.G}, at::kLong, dev), ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
    std::vector<Tensor> out{loss, group_loss, counts, n_valid, ws};
    const uint32_t flags = sum ? LCE_REDUCTION_SUM : 0;
    const uint8_t* keep = static_cast<const uint8_t*>(ptr(r.mask));
    if (grad) {
        out.push_back(like(r.z));
        check(lib.balance_fused(r.G, r.T, r.E, k, r.code, r.z.data_ptr(), r.zg, r.zt, experts.data_ptr(), index_bytes, keep,
                                r.mg, static_cast<float>(grad_scale), go, ptr<float>(loss), ptr<float>(group_loss),
                                ptr<int64_t>(counts), ptr<int64_t>(n_valid), out.back().data_ptr(), ws.data_ptr(), bytes,
                                stream_of(dev), flags),
              "lce_balance_fused");
    } else {
        check(lib.balance_forward(r.G, r.T, r.E, k, r.code, r.z.data_ptr(), r.zg, r.zt, experts.data_ptr(), index_bytes,
                                  keep, r.mg, ptr<float>(loss), ptr<float>(group_loss), ptr<int64_t>(counts),
                                  ptr<int64_t>(n_valid), ws.data_ptr(), bytes, stream_of(dev), flags),
              "lce_balance_forward");
    }
    return out;
}

Tensor balance_backward(const Tensor& logits, const Tensor& counts, const Tensor& n_valid, int64_t slots, const OptTensor& mask,
                        bool sum, double grad_scale, const OptTensor& grad_output) {
    not_traced("balance_backward");
    no_tangent(grad_output, "grad_output");
    const Router r = router_of(logits, mask);
    if (logits.dim() == 3)
        check_shape(counts, {r.G, r.E}, "counts");
    else
        check_shape(counts, {r.E}, "counts");
    check_shape(n_valid, {r.G}, "n_valid");
    for (const Tensor* t : {&counts, &n_valid}) {
        check_type(*t, at::kLong, "counts and n_valid");
        if (!t->is_contiguous()) throw py::type_error("counts and n_valid must be contiguous");
    }
    const at::Device dev = logits.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(counts, dev, "counts");
    on_device(n_valid, dev, "n_valid");
    on_device(r.mask, dev, "mask");
    const float* go = grad_output_of(grad_output, dev);
    const Tensor grad = like(r.z);
    check(lib.balance_backward(r.G, r.T, r.E, slots, r.code, r.z.data_ptr(), r.zg, r.zt, ptr<int64_t>(counts),
                               ptr<int64_t>(n_valid), static_cast<const uint8_t*>(ptr(r.mask)), r.mg,
                               static_cast<float>(grad_scale), go, grad.data_ptr(), stream_of(dev),
                               sum ? LCE_REDUCTION_SUM : 0),
          "lce_balance_backward");
    return grad;
}

// ---------------------------------------------------------------- beams

// scores, tokens, parents and, with eos >= 0, finished
std::vector<Tensor> beam_select(const Tensor& logits_in, const Tensor& scores_in, int64_t n, const OptTensor& finished,
                                int64_t pad, int64_t eos) {
    not_traced("beam_select");
    no_tangent(logits_in, "logits");
    no_tangent(scores_in, "scores");
    const int code = type_code(logits_in, "logits");
    if (logits_in.dim() != 3 || logits_in.numel() == 0)
        throw py::value_error("logits must be [items, beams, V] and not empty, got " + text(logits_in.sizes()));
    const int64_t B = logits_in.size(0), K = logits_in.size(1), V = logits_in.size(2);
    check_shape(scores_in, {B, K}, "scores");
    check_type(scores_in, at::kFloat, "scores");
    OptTensor over;
    if (finished) {
        check_shape(*finished, {B, K}, "finished");
        check_type(*finished, at::kBool, "finished");
        over = finished->contiguous();
    }
    const at::Device dev = logits_in.device();
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(scores_in, dev, "scores");
    on_device(over, dev, "finished");
    // rows evenly spaced (as a last position's logits are in [items * beams, length, V])?
    Tensor logits = logits_in;
    int64_t ld = V;
    if (!logits.is_contiguous()) {
        ld = K > 1 ? logits.stride(1) : B > 1 ? logits.stride(0) : V;
        if (logits.stride(2) != 1 || ld < V || (B > 1 && K > 1 && logits.stride(0) != K * ld)) {
            logits = logits.contiguous();
            ld = V;
        }
    }
    const Tensor scores = scores_in.contiguous();
    size_t bytes = 0;
    check(lib.beam_workspace(B, K, V, n, &bytes), "lce_beam_workspace_size");
    const Tensor ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
    std::vector<Tensor> out{empty({B, n}, at::kFloat, dev), empty({B, n}, at::kLong, dev), empty({B, n}, at::kLong, dev)};
    if (eos >= 0) out.push_back(empty({B, n}, at::kBool, dev));
    check(lib.beam_select(B, K, V, n, code, logits.data_ptr(), ld, ptr<float>(scores),
                          static_cast<const uint8_t*>(ptr(over)), pad, eos, ptr<float>(out[0]), ptr<int64_t>(out[1]),
                          ptr<int64_t>(out[2]), eos >= 0 ? static_cast<uint8_t*>(out[3].data_ptr()) : nullptr,
                          ws.data_ptr(), bytes, stream_of(dev)),
          "lce_beam_select");
    return out;
}

// A state's row as the C ABI describes it, from the strides of src and dst;
// false where that takes more than two strided dimensions.
bool layout_of(const Tensor& src, const Tensor& dst, lce_beam_state_t* s) {
    struct Dim {
        int64_t n, a, b;
    };
    std::vector<Dim> dims;  // outermost first
    for (int64_t i = 1; i < src.dim(); ++i) {
        const Dim d{src.size(i), src.stride(i), dst.stride(i)};
        if (d.n == 1) continue;
        if (!dims.empty() && dims.back().a == d.n * d.a && dims.back().b == d.n * d.b)
            dims.back() = {dims.back().n * d.n, d.a, d.b};
        else
            dims.push_back(d);
    }
    int64_t run = 1;
    if (!dims.empty() && dims.back().a == 1 && dims.back().b == 1) {
        run = dims.back().n;
        dims.pop_back();
    }
    if (dims.size() > 2) return false;
    dims.insert(dims.begin(), 2 - dims.size(), {1, 0, 0});
    const int64_t size = static_cast<int64_t>(src.element_size());
    *s = {src.data_ptr(), dst.data_ptr(), src.stride(0) * size, dst.stride(0) * size,
          dims[0].n, dims[0].a * size, dims[0].b * size, dims[1].n, dims[1].a * size, dims[1].b * size, run * size};
    return true;
}

struct Range {
    uintptr_t first, end;
    int whose;  // 0: a state, 1: an output
    size_t at;  // its place among them
    bool operator<(const Range& o) const { return first < o.first; }
};

Range range_of(const Tensor& t, int whose, size_t at) {
    uintptr_t last = 0;
    for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    const uintptr_t first = reinterpret_cast<uintptr_t>(t.data_ptr());
    return {first, first + (last + 1) * t.element_size(), whose, at};
}

// Whether a state's range of addresses meets an output's.
bool overlap(std::vector<Range> ranges) {
    std::sort(ranges.begin(), ranges.end());
    uintptr_t ends[2] = {0, 0};
    for (const Range& r : ranges) {
        if (r.first < ends[1 - r.whose]) return true;
        ends[r.whose] = std::max(ends[r.whose], r.end);
    }
    return false;
}

// Where a tensor's elements lie, in bytes: n[k] blocks s[k] apart, each of the
// next dimension's, the last of one element; the widest steps first.  Of a
// tensor that is only read (`reads`), what an expanded dimension repeats lies
// where it lies.
struct Places {
    c10::SmallVector<int64_t, 6> n, s, reach;  // reach[k]: from the first to past the last byte of dimensions k, k + 1, ...
    bool nested;  // no dimension's step is shorter than what it steps over: no element lies on another
};

Places places_of(const Tensor& t, bool reads = false) {
    Places p;
    const int64_t size = t.element_size();
    for (int64_t i = 0; i < t.dim(); ++i) {
        if (t.size(i) <= 1 || (reads && t.stride(i) == 0)) continue;
        p.s.push_back(t.stride(i) * size);
        p.n.push_back(t.size(i));
        for (size_t k = p.s.size() - 1; k > 0 && p.s[k - 1] < p.s[k]; --k) {
            std::swap(p.s[k - 1], p.s[k]);
            std::swap(p.n[k - 1], p.n[k]);
        }
    }
    p.reach.assign(p.s.size() + 1, size);
    p.nested = true;
    for (size_t k = p.s.size(); k-- > 0;) {
        p.nested &= p.s[k] >= p.reach[k + 1];
        p.reach[k] = p.reach[k + 1] + (p.n[k] - 1) * p.s[k];
    }
    return p;
}

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }

// Whether an element of a's dimensions i, i + 1, ... and one of b's j, j + 1, ...
// share a byte, b starting d bytes after a; both nested.  Equal steps, as two views
// of one buffer have, leave two distances to look at; of unequal ones the wider is
// gone through, and where that takes too long the two count as sharing.
bool share(const Places& a, size_t i, const Places& b, size_t j, int64_t d, int* budget) {
    if (d >= a.reach[i] || d + b.reach[j] <= 0) return false;
    if (i == a.n.size() && j == b.n.size()) return true;
    if (--*budget < 0) return true;
    const int64_t sa = i < a.n.size() ? a.s[i] : 0, sb = j < b.n.size() ? b.s[j] : 0;
    if (sa == sb) {
        // block v of b starts (q + v - u) sa + r bytes after block u of a, and a block reaches no further than sa
        const int64_t q = floor_div(d, sa), r = d - q * sa;
        const int64_t least = -(b.n[j] - 1), most = a.n[i] - 1;  // of u - v
        return (q >= least && q <= most && share(a, i + 1, b, j + 1, r, budget)) ||
               (q + 1 >= least && q + 1 <= most && share(a, i + 1, b, j + 1, r - sa, budget));
    }
    if (sa < sb) return share(b, j, a, i, -d, budget);
    int64_t u = floor_div(d - a.reach[i + 1], sa) + 1;
    if (u < 0) u = 0;
    for (; u < a.n[i] && u * sa < d + b.reach[j]; ++u)
        if (share(a, i + 1, b, j, d - u * sa, budget)) return true;
    return false;
}

// No output lies on another one, or on itself.
void outputs_apart(const std::vector<Tensor>& out, std::vector<Range> ranges) {
    for (size_t i = 0; i < out.size(); ++i) {
        const Tensor& t = out[i];
        int64_t reach = t.numel() ? 1 : 0;
        bool nested = true;  // in the order of its dimensions, as nearly all are
        for (int64_t k = t.dim(); k-- > 0 && reach;) {
            if (t.size(k) == 1) continue;
            nested &= t.stride(k) >= reach;
            reach += (t.size(k) - 1) * t.stride(k);
        }
        if (!nested && !places_of(t).nested)
            throw py::value_error("out[" + std::to_string(i) + "] overlaps itself: strides " + text(t.strides()));
    }
    std::sort(ranges.begin(), ranges.end());
    std::vector<const Range*> open;  // outputs that reach past the current one's start
    std::vector<std::optional<Places>> places;
    auto at = [&](const Range& r) -> const Places& {
        places.resize(out.size());
        if (!places[r.at]) places[r.at] = places_of(out[r.at]);
        return *places[r.at];
    };
    for (const Range& r : ranges) {
        if (!r.whose) continue;
        open.erase(std::remove_if(open.begin(), open.end(), [&](const Range* o) { return o->end <= r.first; }), open.end());
        for (const Range* o : open) {
            int budget = 1 << 16;
            if (share(at(*o), 0, at(r), 0, static_cast<int64_t>(r.first - o->first), &budget))
                throw py::value_error("out[" + std::to_string(o->at) + "] overlaps out[" + std::to_string(r.at) + "]");
        }
        open.push_back(&r);
    }
}

// Whether an element of an output is one of a state's, whose ranges may meet.
bool states_meet(const std::vector<Tensor>& states, const std::vector<Tensor>& out, const std::vector<Range>& ranges) {
    for (const Range& a : ranges)
        for (const Range& b : ranges) {
            if (a.whose || !b.whose || a.end <= b.first || b.end <= a.first) continue;
            const Places x = places_of(states[a.at], true), y = places_of(out[b.at]);
            int budget = 1 << 16;
            if (!x.nested || !y.nested || share(x, 0, y, 0, static_cast<int64_t>(b.first - a.first), &budget)) return true;
        }
    return false;
}

std::vector<Tensor> beam_reorder(const std::vector<Tensor>& states, const Tensor& parents_in,
                                 std::optional<std::vector<Tensor>> given, const OptTensor& status) {
    not_traced("beam_reorder");
    if (parents_in.dim() != 2 || parents_in.scalar_type() != at::kLong || parents_in.numel() == 0)
        throw py::value_error("parents must be int64 [items, n] and not empty");
    const int64_t B = parents_in.size(0), n = parents_in.size(1);
    if (states.empty()) return {};
    if (states[0].dim() == 0 || states[0].size(0) == 0 || states[0].size(0) % B)
        throw py::value_error("a state's first dimension must be a multiple of the " + std::to_string(B) + " items");
    const int64_t rows = states[0].size(0);
    const at::Device dev = states[0].device();
    if (given && given->size() != states.size())
        throw py::value_error(std::to_string(states.size()) + " states, but " + std::to_string(given->size()) + " outputs");
    std::vector<Tensor> out, copies;  // copies live until the launch is enqueued
    std::vector<lce_beam_state_t> moves;
    std::vector<Range> ranges;
    // many of these are views, whose answer takes 35 ns each: not outside a dual level
    const bool dual = torch::autograd::ForwardADLevel::try_get_by_idx(0) != nullptr;
    for (size_t i = 0; i < states.size(); ++i) {
        Tensor a = states[i];
        if (dual) no_tangent(a, "a state");
        if (a.dim() == 0 || a.size(0) != rows)
            throw py::value_error("states must have " + std::to_string(rows) + " rows each, states[" + std::to_string(i) +
                                  "] has shape " + text(a.sizes()));
        std::vector<int64_t> shape = a.sizes().vec();
        shape[0] = B * n;
        if (a.device() != dev) throw py::value_error("states and outputs must be on " + dev.str());
        if (a.is_conj() || a.is_neg()) {  // memory that stands for other values
            a = a.resolve_conj().resolve_neg();
            copies.push_back(a);
        }
        Tensor b;
        if (given) {
            b = (*given)[i];
            if (dual) no_tangent(b, "an output");
            check_shape(b, shape, ("out[" + std::to_string(i) + "]").c_str());
            check_type(b, a.scalar_type(), ("out[" + std::to_string(i) + "]").c_str());
            if (b.device() != dev) throw py::value_error("states and outputs must be on " + dev.str());
            if (b.is_conj() || b.is_neg()) throw py::value_error("out[" + std::to_string(i) + "] is a conjugate or negative view");
        } else {
            b = empty(shape, a.scalar_type(), dev);
        }
        out.push_back(b);
        if (a.numel() == 0) continue;
        if (given) {
            ranges.push_back(range_of(a, 0, i));
            ranges.push_back(range_of(b, 1, i));
        }
        lce_beam_state_t s;
        if (!layout_of(a, b, &s)) {
            a = a.contiguous();
            copies.push_back(a);
            if (!layout_of(a, b, &s)) throw py::value_error("an output has more than two strided dimensions: " + text(b.strides()));
        }
        moves.push_back(s);
    }
    if (overlap(ranges) && states_meet(states, out, ranges)) throw py::value_error("out overlaps the states");
    if (given) outputs_apart(out, std::move(ranges));
    on_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    on_device(parents_in, dev, "parents");
    const Tensor parents = parents_in.contiguous();
    check(lib.beam_reorder(B, rows / B, n, ptr<int64_t>(parents), moves.data(), static_cast<int64_t>(moves.size()),
                           ptr(status), stream_of(dev)),
          "lce_beam_reorder");
    return out;
}

// ---- seen by the tests

py::object layout_for_test(const Tensor& src, const Tensor& dst) {
    lce_beam_state_t s;
    if (!layout_of(src, dst, &s)) return py::none();
    return py::make_tuple(s.n1, s.src1, s.dst1, s.n2, s.src2, s.dst2, s.run_bytes);
}

bool overlap_for_test(const std::vector<std::tuple<uintptr_t, uintptr_t, int>>& ranges) {
    std::vector<Range> r;
    for (const auto& [first, end, whose] : ranges) r.push_back({first, end, whose, 0});
    return overlap(std::move(r));
}

}  // namespace

PYBIND11_MODULE(_lce_torch, m) {
    m.def("init", &init);
    m.def("norm_forward", &norm_forward);
    m.def("norm_backward", &norm_backward);
    m.def("balance_call", &balance_call);
    m.def("balance_backward", &balance_backward);
    m.def("beam_select", &beam_select);
    m.def("beam_reorder", &beam_reorder);
    m.def("layout", &layout_for_test);
    m.def("overlap", &overlap_for_test);
    bind_rows(m);
}
