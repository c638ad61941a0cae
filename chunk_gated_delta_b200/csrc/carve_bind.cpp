// Host side of the Python calls of include/carve_mixers.h (mixers.py documents them): checks of the
// tensors, allocation of what the caller did not give, and the C call on the right device and stream.
//
// In C++ because these calls are short: a decoding step's kernel takes 3 us, and the same checks and
// allocations took 8 us in Python around a 4 us launch (a small training call 53 us around 14 us).
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <pybind11/stl.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <climits>
#include <sstream>

#include "../../include/carve_mixers.h"

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

namespace {

const char *dtype_name(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kDouble: return "torch.float64";
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        default: return c10::toString(t);
    }
}
std::string shape_name(at::IntArrayRef s) {
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << s[i] << (i + 1 < s.size() ? ", " : s.size() == 1 ? "," : "");
    o << ")";
    return o.str();
}

[[noreturn]] void complain(const Tensor &like, const char *name, const Tensor &x, at::IntArrayRef shape, at::ScalarType dtype) {
    std::ostringstream o;
    o << name;
    if (x.device() != like.device()) {
        o << " is on " << x.device() << ", q (or k) on " << like.device();
        throw py::value_error(o.str());
    }
    if (x.scalar_type() != dtype) {
        o << " must be " << dtype_name(dtype) << ", got " << dtype_name(x.scalar_type());
        throw py::type_error(o.str());
    }
    if (x.sizes() != shape) {
        o << " must have shape " << shape_name(shape) << ", got " << shape_name(x.sizes());
        throw py::value_error(o.str());
    }
    o << " must be contiguous";
    throw py::value_error(o.str());
}
// x has this shape and dtype, is contiguous and on the device of `like`
void want(const Tensor &like, const char *name, const Tensor &x, at::IntArrayRef shape, at::ScalarType dtype) {
    if (x.device() != like.device() || x.scalar_type() != dtype || x.sizes() != shape || !x.is_contiguous())
        complain(like, name, x, shape, dtype);
}
void want(const Tensor &like, const char *name, const Opt &x, at::IntArrayRef shape, at::ScalarType dtype) {
    if (x) want(like, name, *x, shape, dtype);
}
void want_cuda(const Tensor &like) {
    if (like.is_cuda()) return;
    std::ostringstream o;
    o << "tensors must be on a CUDA device, got " << like.device();
    throw py::value_error(o.str());
}
int io_of(const Tensor &x) {
    if (x.scalar_type() == at::kBFloat16) return CARVE_IO_BF16;
    if (x.scalar_type() == at::kFloat) return CARVE_IO_FP32;
    throw py::type_error(std::string("q must be float32 or bfloat16, got ") + dtype_name(x.scalar_type()));
}
void want_rank(const Tensor &x, int64_t n, const char *what) {
    if (x.dim() == n) return;
    std::ostringstream o;
    o << what << " must have " << n << " dimensions, got shape " << shape_name(x.sizes());
    throw py::value_error(o.str());
}
void want_heads(int64_t few, int64_t many, const char *what) {
    if (few >= 1 && many % few == 0) return;
    std::ostringstream o;
    o << what << ": " << many << " heads are not a multiple of " << few;
    throw py::value_error(o.str());
}
int small(int64_t n) {
    if (n > INT_MAX) throw py::value_error("a dimension exceeds 2^31 - 1");
    return (int)n;
}

// leading dimensions of a token tensor, and what they say of the sequences
struct Lead {
    at::DimVector dims;
    int B, T;
    int64_t rows;
    bool packed;
    Lead(const Tensor &x, const Opt &cu) : packed(cu.has_value()) {
        if (!packed) {
            want_rank(x, 4, "q");
            dims = {x.size(0), x.size(1)};
            B = small(x.size(0));
            T = small(x.size(1));
            rows = x.size(0) * x.size(1);
            return;
        }
        want_rank(x, 3, "packed q");
        want_rank(*cu, 1, "cu_seqlens");
        if (cu->scalar_type() != at::kInt)
            throw py::type_error(std::string("cu_seqlens must be torch.int32, got ") + dtype_name(cu->scalar_type()));
        if (cu->device() != x.device() || !cu->is_contiguous())
            throw py::value_error("cu_seqlens must be a contiguous tensor on the device of the tokens");
        if (cu->numel() < 2) throw py::value_error("cu_seqlens needs at least two offsets");
        dims = {x.size(0)};
        B = small(cu->numel() - 1);
        T = 0;
        rows = x.size(0);
    }
    at::DimVector with(int64_t a) const {
        at::DimVector d = dims;
        d.push_back(a);
        return d;
    }
    at::DimVector with(int64_t a, int64_t b) const {
        at::DimVector d = with(a);
        d.push_back(b);
        return d;
    }
};

void *ptr(const Tensor &x) { return x.data_ptr(); }
void *ptr(const Opt &x) { return x ? x->data_ptr() : nullptr; }
template <class T>
T *as(const Tensor &x) { return static_cast<T *>(x.data_ptr()); }
template <class T>
T *as(const Opt &x) { return x ? static_cast<T *>(x->data_ptr()) : nullptr; }

void raise(const char *fn, int rc) {
    if (rc == CARVE_OK) return;
    const py::object type = py::module_::import("chunk_gated_delta_b200").attr("CarveError");
    PyErr_SetObject(type.ptr(), type(fn, rc).ptr());
    throw py::error_already_set();
}

// The device of `like` and the stream of the call current: the caller's stream or the device's current one.  Stands
// before the call's allocations, so that what it allocates belongs to the stream that uses it (as within
// torch.cuda.stream): scratch is released when the call returns, and the memory may then serve other
// streams only behind this one's work.
struct On {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard current;
    void *stream;
    On(const Tensor &like, const py::object &s) : device(like.device()) {
        if (s.is_none()) {
            stream = c10::cuda::getCurrentCUDAStream(like.device().index()).stream();
            return;
        }
        const c10::Device d = s.attr("device").cast<c10::Device>();
        if (d != like.device()) {
            std::ostringstream o;
            o << "the stream is on " << d << ", the tensors on " << like.device();
            throw py::value_error(o.str());
        }
        stream = reinterpret_cast<void *>(s.attr("cuda_stream").cast<uintptr_t>());
        current.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), d.index()));
    }
};

// a buffer of `n` bytes: the caller's, checked, or a new one
Tensor buffer(const char *name, const Opt &given, const char *sized_by, size_t n, const Tensor &like) {
    if (n == 0) raise(sized_by, CARVE_ERR_INVALID_ARG);
    if (!given) return at::empty({(int64_t)n}, like.options().dtype(at::kByte));
    if (given->device() != like.device() || !given->is_contiguous()) {
        std::ostringstream o;
        o << name << " must be a contiguous tensor on " << like.device();
        throw py::value_error(o.str());
    }
    if ((size_t)given->nbytes() < n) {
        std::ostringstream o;
        o << name << " holds " << given->nbytes() << " bytes, " << n << " are needed";
        throw py::value_error(o.str());
    }
    return *given;
}

py::dict copy_of(const py::object &out) {
    return out.is_none() ? py::dict() : py::reinterpret_steal<py::dict>(PyDict_Copy(py::dict(out).ptr()));
}
// out[key], if there is one; None counts as none
Opt given(const py::dict &out, const char *key) {
    const py::str k(key);
    if (!out.contains(k) || out[k].is_none()) return std::nullopt;
    if (!THPVariable_Check(py::object(out[k]).ptr())) throw py::type_error(std::string(key) + " must be a tensor");
    return out[k].cast<Tensor>();
}
// a result: the caller's, or a new tensor that is put there
Tensor result(py::dict &out, const char *key, at::IntArrayRef shape, const at::TensorOptions &options) {
    if (const Opt x = given(out, key)) return *x;
    Tensor x = at::empty(shape, options);
    out[py::str(key)] = x;
    return x;
}

// ---- the scalar-gated delta rule ----------------------------------------------------------
struct Gdr {
    Lead lead;
    carve_gdr_dims d;
    at::ScalarType dt;
    at::DimVector state, gates;
    Gdr(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &w, const Opt &A_dec, const Opt &tau,
        const Opt &cu, int io)
        : lead(q, cu), dt(q.scalar_type()) {
        const int64_t n = lead.dims.size(), Hk = q.size(n), dk = q.size(n + 1);
        want_rank(v, n + 2, "v");
        const int64_t Hv = v.size(n), dv = v.size(n + 1);
        want_heads(Hk, Hv, "value heads on key heads");
        gates = lead.with(Hv);
        const at::DimVector keys = lead.with(Hk, dk);
        want(q, "q", q, keys, dt);
        want(q, "k", k, keys, dt);
        want(q, "v", v, lead.with(Hv, dv), dt);
        want(q, "g_logit", g, gates, dt);
        want(q, "w_logit", w, gates, dt);
        want(q, "A_dec", A_dec, {Hv}, at::kFloat);
        want(q, "tau", tau, {Hv}, at::kFloat);
        if (cu) want(q, "cu_seqlens", *cu, cu->sizes(), at::kInt);
        want_cuda(q);
        d = carve_gdr_dims{lead.B, lead.T, small(Hk), small(Hv), small(dk), small(dv), io, lead.rows};
        state = {lead.B, Hv, dv, dk};
    }
};

py::dict gdr_fwd(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &w, const Opt &A_dec,
                 const Opt &tau, const Opt &S0, const Opt &cu, bool save, const py::object &out_, const Opt &ws_,
                 const py::object &stream) {
    const int io = io_of(q);
    const Gdr c(q, k, v, g, w, A_dec, tau, cu, io);
    const bool packed = c.lead.packed;
    const On on(q, stream);
    py::dict out = copy_of(out_);
    const Tensor o = result(out, "o", v.sizes(), v.options());
    const Tensor S = result(out, "S_final", c.state, v.options().dtype(at::kFloat));
    want(q, "S0", S0, c.state, at::kFloat);
    want(q, "o", o, v.sizes(), c.dt);
    want(q, "S_final", S, c.state, at::kFloat);
    Opt saved, ws;
    if (save) {
        saved = buffer("saved", given(out, "saved"), "carve_gdr_saved_bytes", carve_gdr_saved_bytes(&c.d, packed), q);
        out["saved"] = *saved;
    }
    if (!save || ws_)
        ws = buffer("workspace", ws_, "carve_gdr_fwd_workspace_bytes", carve_gdr_fwd_workspace_bytes(&c.d, packed), q);
    raise("carve_gdr_fwd", carve_gdr_fwd(&c.d, as<int32_t>(cu), ptr(q), ptr(k), ptr(v), ptr(g), ptr(w), as<float>(A_dec),
                                         as<float>(tau), as<float>(S0), ptr(o), as<float>(S), ptr(saved), ptr(ws), on.stream));
    return out;
}

py::dict gdr_bwd(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &w, const Tensor &saved,
                 const Tensor &dO, const Opt &A_dec, const Opt &tau, const Opt &dS, const Opt &cu, bool want_dS0,
                 const py::object &out_, const Opt &ws_, const py::object &stream) {
    const int io = io_of(q);
    const Gdr c(q, k, v, g, w, A_dec, tau, cu, io);
    const bool packed = c.lead.packed;
    const On on(q, stream);
    const auto f32 = v.options().dtype(at::kFloat);
    py::dict out = copy_of(out_);
    auto grad = [&](const char *key, at::IntArrayRef shape, const at::TensorOptions &opt) {
        Tensor x = result(out, key, shape, opt);
        want(q, key, x, shape, c10::typeMetaToScalarType(opt.dtype()));
        return x;
    };
    want(q, "dO", dO, v.sizes(), c.dt);
    want(q, "dS_final", dS, c.state, at::kFloat);
    const Tensor dq = grad("dq", q.sizes(), q.options()), dk = grad("dk", k.sizes(), q.options()),
                 dv = grad("dv", v.sizes(), q.options()), dg = grad("dg_logit", c.gates, q.options()),
                 dw = grad("dw_logit", c.gates, q.options());
    Opt dS0, dA, dt;
    if (want_dS0) dS0 = grad("dS0", c.state, f32);
    if (A_dec) dA = grad("dA_dec", {c.d.Hv}, f32);
    if (tau) dt = grad("dtau", {c.d.Hv}, f32);
    buffer("saved", saved, "carve_gdr_saved_bytes", carve_gdr_saved_bytes(&c.d, packed), q);
    const Tensor ws = buffer("workspace", ws_, "carve_gdr_bwd_workspace_bytes", carve_gdr_bwd_workspace_bytes(&c.d, packed), q);
    raise("carve_gdr_bwd",
          carve_gdr_bwd(&c.d, as<int32_t>(cu), ptr(q), ptr(k), ptr(v), ptr(g), ptr(w), as<float>(A_dec), as<float>(tau), ptr(saved),
                        ptr(dO), as<float>(dS), ptr(dq), ptr(dk), ptr(dv), ptr(dg), ptr(dw), as<float>(dA), as<float>(dt),
                        as<float>(dS0), ptr(ws), on.stream));
    return out;
}

Tensor gdr_step(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &w, const Tensor &S,
                const Opt &A_dec, const Opt &tau, const Opt &o_, const py::object &stream) {
    const int io = io_of(q);
    want_rank(q, 3, "q");
    want_rank(v, 3, "v");
    const int64_t B = q.size(0), Hk = q.size(1), dk = q.size(2), Hv = v.size(1), dv = v.size(2);
    want_heads(Hk, Hv, "value heads on key heads");
    const at::ScalarType dt = q.scalar_type();
    want(q, "q", q, q.sizes(), dt);
    want(q, "k", k, q.sizes(), dt);
    want(q, "v", v, {B, Hv, dv}, dt);
    want(q, "g_logit", g, {B, Hv}, dt);
    want(q, "w_logit", w, {B, Hv}, dt);
    want(q, "S", S, {B, Hv, dv, dk}, at::kFloat);
    want(q, "A_dec", A_dec, {Hv}, at::kFloat);
    want(q, "tau", tau, {Hv}, at::kFloat);
    want(q, "o", o_, v.sizes(), dt);
    want_cuda(q);
    const On on(q, stream);
    const Tensor o = o_ ? *o_ : at::empty(v.sizes(), v.options());
    const carve_gdr_dims d{small(B), 1, small(Hk), small(Hv), small(dk), small(dv), io, 0};
    raise("carve_gdr_step", carve_gdr_step(&d, ptr(q), ptr(k), ptr(v), ptr(g), ptr(w), as<float>(A_dec), as<float>(tau), as<float>(S),
                                           ptr(o), on.stream));
    return o;
}

// ---- sliding-window attention with sink tokens ----------------------------------------------
void want_window(int64_t window, int64_t sinks) {
    if (window >= 1 && window <= INT_MAX && sinks >= 0 && sinks <= INT_MAX) return;
    std::ostringstream o;
    o << "window must be 1 .. 2^31 - 1 and sinks 0 .. 2^31 - 1, got " << window << " and " << sinks;
    throw py::value_error(o.str());
}
float scale_of(const std::optional<double> &scale, int64_t d) {
    return scale ? (float)*scale : (float)(1.0 / std::sqrt((double)d));
}

struct Swa {
    Lead lead;
    carve_swa_dims d;
    at::ScalarType dt;
    Swa(const Tensor &q, const Tensor &k, const Tensor &v, int64_t window, int64_t sinks, const std::optional<double> &scale,
        const Opt &cu, int io)
        : lead(q, cu), dt(q.scalar_type()) {
        const int64_t n = lead.dims.size(), Hq = q.size(n), D = q.size(n + 1);
        want_rank(k, n + 2, "k");
        const int64_t Hkv = k.size(n);
        want_heads(Hkv, Hq, "query heads on key heads");
        const at::DimVector kv = lead.with(Hkv, D);
        want(q, "q", q, q.sizes(), dt);
        want(q, "k", k, kv, dt);
        want(q, "v", v, kv, dt);
        want_cuda(q);
        d = carve_swa_dims{lead.B, lead.T, small(Hq), small(Hkv), small(D), (int)window, (int)sinks, io, scale_of(scale, D), lead.rows};
    }
};

py::dict swa_fwd(const Tensor &q, const Tensor &k, const Tensor &v, int64_t window, int64_t sinks, std::optional<double> scale,
                 const Opt &cu, bool want_lse, const py::object &out_, const py::object &stream) {
    want_window(window, sinks);
    const int io = io_of(q);
    const Swa c(q, k, v, window, sinks, scale, cu, io);
    const On on(q, stream);
    py::dict out = copy_of(out_);
    const Tensor o = result(out, "o", q.sizes(), q.options());
    Opt lse = given(out, "lse");
    const at::IntArrayRef rows = q.sizes().slice(0, q.dim() - 1);
    if (want_lse && !lse) {
        lse = at::empty(rows, q.options().dtype(at::kFloat));
        out["lse"] = *lse;
    }
    want(q, "o", o, q.sizes(), c.dt);
    want(q, "lse", lse, rows, at::kFloat);
    raise("carve_swa_fwd", carve_swa_fwd(&c.d, as<int32_t>(cu), ptr(q), ptr(k), ptr(v), ptr(o), want_lse ? as<float>(lse) : nullptr,
                                         on.stream));
    return out;
}

py::dict swa_bwd(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &o, const Tensor &lse, const Tensor &dO,
                 int64_t window, int64_t sinks, std::optional<double> scale, const Opt &cu, const py::object &out_, const Opt &ws_,
                 const py::object &stream) {
    want_window(window, sinks);
    const int io = io_of(q);
    const Swa c(q, k, v, window, sinks, scale, cu, io);
    const On on(q, stream);
    py::dict out = copy_of(out_);
    const Tensor dq = result(out, "dq", q.sizes(), q.options()), dk = result(out, "dk", k.sizes(), k.options()),
                 dv = result(out, "dv", v.sizes(), v.options());
    want(q, "o", o, q.sizes(), c.dt);
    want(q, "dO", dO, q.sizes(), c.dt);
    want(q, "lse", lse, q.sizes().slice(0, q.dim() - 1), at::kFloat);
    want(q, "dq", dq, q.sizes(), c.dt);
    want(q, "dk", dk, k.sizes(), c.dt);
    want(q, "dv", dv, k.sizes(), c.dt);
    const Tensor ws =
        buffer("workspace", ws_, "carve_swa_bwd_workspace_bytes", carve_swa_bwd_workspace_bytes(&c.d, c.lead.packed), q);
    raise("carve_swa_bwd", carve_swa_bwd(&c.d, as<int32_t>(cu), ptr(q), ptr(k), ptr(v), ptr(o), as<float>(lse), ptr(dO), ptr(dq),
                                         ptr(dk), ptr(dv), ptr(ws), on.stream));
    return out;
}

void swa_fill(const Tensor &k, const Tensor &v, const Tensor &kc, const Tensor &vc, int64_t window, int64_t sinks, const Opt &cu,
              const py::object &stream) {
    want_window(window, sinks);
    const int io = io_of(k);
    const Swa c(k, k, v, window, sinks, 1.0, cu, io);
    const On on(k, stream);
    const at::DimVector slots = {c.d.B, sinks + window, c.d.Hkv, c.d.d};
    want(k, "k_cache", kc, slots, c.dt);
    want(k, "v_cache", vc, slots, c.dt);
    raise("carve_swa_fill", carve_swa_fill(&c.d, as<int32_t>(cu), ptr(k), ptr(v), ptr(kc), ptr(vc), on.stream));
}

Tensor swa_step(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &kc, const Tensor &vc, const Tensor &pos,
                int64_t window, int64_t sinks, std::optional<double> scale, const Opt &o_, const py::object &stream) {
    want_window(window, sinks);
    const int io = io_of(q);
    want_rank(q, 3, "q");
    want_rank(k, 3, "k");
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
    want_heads(Hkv, Hq, "query heads on key heads");
    const at::ScalarType dt = q.scalar_type();
    want(q, "q", q, q.sizes(), dt);
    want(q, "k", k, {B, Hkv, D}, dt);
    want(q, "v", v, {B, Hkv, D}, dt);
    want(q, "pos", pos, {B}, at::kLong);
    want(q, "o", o_, q.sizes(), dt);
    want(q, "k_cache", kc, {B, sinks + window, Hkv, D}, dt);
    want(q, "v_cache", vc, {B, sinks + window, Hkv, D}, dt);
    want_cuda(q);
    const On on(q, stream);
    const Tensor o = o_ ? *o_ : at::empty(q.sizes(), q.options());
    const carve_swa_dims d{small(B), 1, small(Hq), small(Hkv), small(D), (int)window, (int)sinks, io, scale_of(scale, D), 0};
    raise("carve_swa_step", carve_swa_step(&d, ptr(q), ptr(k), ptr(v), ptr(kc), ptr(vc), as<int64_t>(pos), ptr(o), on.stream));
    return o;
}

}  // namespace

PYBIND11_MODULE(_carve_bind, m) {
    m.def("gdr_fwd", &gdr_fwd);
    m.def("gdr_bwd", &gdr_bwd);
    m.def("gdr_step", &gdr_step);
    m.def("swa_fwd", &swa_fwd);
    m.def("swa_bwd", &swa_bwd);
    m.def("swa_fill", &swa_fill);
    m.def("swa_step", &swa_step);
}
