// binding.cpp -- torch tensors into the C ABI of include/gtr_ssm.h and include/gtr_norm.h, for
// ssm.py and norm.py: checks of tensor metadata, allocation of absent outputs and workspaces on the
// current stream, and the call.  (A single token's kernels take a few microseconds; the same checks in
// Python took twenty.)  Every function takes its arguments by position and returns the outputs, or
// the library's status where the call failed.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <array>
#include <string>
#include <vector>

#include "../../include/gtr_norm.h"
#include "../../include/gtr_ssm.h"

namespace {

using at::Tensor;
using Sizes = at::IntArrayRef;

[[noreturn]] void refuse(const std::string &why) {   // ValueError
    throw c10::ValueError({__func__, __FILE__, (uint32_t)__LINE__}, why);
}

std::string show(Sizes s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

const Tensor *tensor_or_none(PyObject *o, const char *name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor or None");
    return &THPVariable_Unpack(o);
}
const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject *o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw python_error();
    return t != 0;
}
int small(PyObject *o, const char *name) {
    const long long v = integer(o);
    if (v < -0x7fffffffLL || v > 0x7fffffffLL) refuse(std::string(name) + " is out of range");
    return (int)v;
}

// The tensor lives on the current device (the library launches there).
int device_of(const Tensor &t, const char *name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    const int cur = c10::cuda::current_device();
    if (t.get_device() != cur)
        refuse(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", but the current CUDA device is cuda:" +
               std::to_string(cur));
    return cur;
}

struct Call {
    at::ScalarType type;
    int dtype, dev;
    const Tensor &like;

    Call(const Tensor &x, const char *name) : type(x.scalar_type()), dtype(0), dev(0), like(x) {
        if (type != at::kHalf && type != at::kBFloat16) refuse(std::string(name) + " must be float16 or bfloat16");
        dtype = type == at::kHalf ? GTR_F16 : GTR_BF16;
        dev = device_of(x, name);
    }
    void on_device(const Tensor &t, const char *name) const {
        if (!t.is_cuda() || t.get_device() != dev) device_of(t, name);
    }
    // A [B, N, cols] activation with evenly spaced rows: the elements between them.
    long long rows(const Tensor &t, const char *name, int64_t B, int64_t N, int64_t cols) const {
        if (t.sizes() != Sizes({B, N, cols})) refuse(std::string(name) + " must be " + show({B, N, cols}) + ", not " + show(t.sizes()));
        if (t.scalar_type() != type) refuse(std::string(name) + " must have the type of the other activations");
        on_device(t, name);
        if (t.is_contiguous()) return cols;
        if (t.numel() == 0) return 0;
        const int64_t sb = t.stride(0), sn = t.stride(1), sc = t.stride(2);
        if (cols > 1 && sc != 1) refuse(std::string(name) + "'s channels must be contiguous");
        const int64_t ld = N > 1 ? sn : B > 1 ? sb : cols;
        if (ld < cols || (B > 1 && sb != N * ld)) refuse(std::string(name) + "'s token rows must be evenly spaced and must not overlap");
        return ld;
    }
    template <typename P = void>
    P *dense(const Tensor *t, const char *name, Sizes sizes, at::ScalarType ty, bool required) const {
        if (t == nullptr) {
            if (required) refuse(std::string(name) + " is required");
            return nullptr;
        }
        if (t->scalar_type() != ty || t->sizes() != sizes || !t->is_contiguous())
            refuse(std::string(name) + " must be a contiguous " + c10::toString(ty) + " tensor " + show(sizes));
        on_device(*t, name);
        return static_cast<P *>(t->data_ptr());
    }
    Tensor make(Sizes sizes, at::ScalarType ty) const {
        return at::empty(sizes, at::TensorOptions().dtype(ty).device(like.device()));
    }
    // The caller's workspace or a new one of `need` bytes.
    void *workspace(PyObject *o, size_t need, Tensor &keep, size_t &bytes) const {
        bytes = 0;
        if (need == 0) return nullptr;
        if (o == Py_None) {
            keep = make({(int64_t)need}, at::kByte);
        } else {
            keep = tensor(o, "workspace");
            on_device(keep, "workspace");
            if (!keep.is_contiguous()) refuse("workspace must be contiguous");
        }
        bytes = keep.nbytes();
        return keep.data_ptr();
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

// An output given, wanted (True) or left out (None).
Tensor output(PyObject *o, const Call &c, Sizes sizes, at::ScalarType ty, const char *name) {
    if (o == Py_None) return Tensor();
    if (o == Py_True) return c.make(sizes, ty);
    return tensor(o, name);
}
PyObject *wrap(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject *result(int status, std::initializer_list<const Tensor *> outs) {
    if (status != GTR_OK) return PyLong_FromLong(status);
    PyObject *r = PyTuple_New((Py_ssize_t)outs.size());
    if (r == nullptr) throw python_error();
    Py_ssize_t i = 0;
    for (const Tensor *t : outs) PyTuple_SET_ITEM(r, i++, wrap(*t));
    return r;
}
void count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse("wrong number of arguments");
}
// The gradients given (a tuple of n tensors or None), or an empty list.
std::vector<Tensor> given(PyObject *o, Py_ssize_t n) {
    std::vector<Tensor> g;
    if (o == Py_None) return g;
    PyObject *seq = PySequence_Fast(o, "grads must be a tuple of tensors");
    if (seq == nullptr) throw python_error();
    THPObjectPtr hold(seq);
    if (PySequence_Fast_GET_SIZE(seq) != n) refuse("grads must hold " + std::to_string(n) + " tensors (or None)");
    for (Py_ssize_t i = 0; i < n; ++i) {
        const Tensor *t = tensor_or_none(PySequence_Fast_GET_ITEM(seq, i), "a gradient");
        g.push_back(t ? *t : Tensor());
    }
    return g;
}
const Tensor *at_or_none(const Tensor &t) { return t.defined() ? &t : nullptr; }

// ------------------------------------------------------------------ convolution
struct Conv {
    const Tensor &x, &w;
    const Tensor *bias, *init;
    Call c;
    int64_t B, N, D, K;
    gtr_conv_t a{};

    Conv(PyObject *x_, PyObject *w_, PyObject *bias_, PyObject *init_, PyObject *H, PyObject *W, PyObject *dir, PyObject *act)
        : x(tensor(x_, "x")), w(tensor(w_, "w")), bias(tensor_or_none(bias_, "bias")),
          init(tensor_or_none(init_, "init_state")), c(x, "x") {
        if (x.dim() != 3) refuse("x must be [B, N, channels]");
        if (w.dim() != 2) refuse("w must be [D, K]");
        B = x.size(0), N = x.size(1), D = x.size(2), K = w.size(1);
        const int h = small(H, "Hgrid"), v = small(W, "Wgrid");
        if (N != (int64_t)h * v) refuse("N=" + std::to_string(N) + " does not match the grid " + std::to_string(h) + "x" + std::to_string(v));
        if (B > 0x7fffffff || D > 0x7fffffff || K > 0x7fffffff) refuse("x is too large");
        a.B = (int)B, a.Hgrid = h, a.Wgrid = v, a.D = (int)D, a.K = (int)K;
        a.direction = small(dir, "direction");
        a.dtype = c.dtype;
        a.activation = small(act, "activation");
        a.ldx = c.rows(x, "x", B, N, D);
        a.x = x.data_ptr();
        a.w = c.dense<float>(&w, "w", {D, K}, at::kFloat, true);
        a.bias = c.dense<float>(bias, "bias", {D}, at::kFloat, false);
        a.init_state = c.dense(init, "init_state", {B, K - 1, D}, c.type, false);
    }
    std::array<int64_t, 3> state() const { return {B, K > 0 ? K - 1 : 0, D}; }
};

// x, w, bias, init_state, out (or None), final_state (or True, None), Hgrid, Wgrid, direction, activation
PyObject *conv_fwd(PyObject *, PyObject *const *p, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 10);
    const Conv v(p[0], p[1], p[2], p[3], p[6], p[7], p[8], p[9]);
    const Tensor out = output(p[4] == Py_None ? Py_True : p[4], v.c, {v.B, v.N, v.D}, v.c.type, "out");
    const auto st = v.state();
    const Tensor fin = output(p[5], v.c, st, v.c.type, "final_state");
    return result(gtr_causal_conv_fwd(&v.a, v.c.dense(&out, "out", {v.B, v.N, v.D}, v.c.type, true),
                                      v.c.dense(at_or_none(fin), "final_state", st, v.c.type, false), v.c.stream()),
                  {&out, &fin});
    END_HANDLE_TH_ERRORS
}

// x, w, d_out, bias, init_state, d_final_state, workspace, grads, want_init_grad, Hgrid, Wgrid, direction, activation
PyObject *conv_bwd(PyObject *, PyObject *const *p, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 13);
    const Conv v(p[0], p[1], p[3], p[4], p[9], p[10], p[11], p[12]);
    const Call &c = v.c;
    const Tensor &dy = tensor(p[2], "d_out");
    const long long ld = c.rows(dy, "d_out", v.B, v.N, v.D);
    const auto st = v.state();
    const void *df = c.dense(tensor_or_none(p[5], "d_final_state"), "d_final_state", st, c.type, false);
    std::vector<Tensor> g = given(p[7], 4);
    if (g.empty())
        g = {c.make({v.B, v.N, v.D}, c.type), c.make({v.D, v.K}, at::kFloat),
             v.bias ? c.make({v.D}, at::kFloat) : Tensor(), truth(p[8]) ? c.make(st, c.type) : Tensor()};
    Tensor keep;
    size_t bytes;
    void *ws = c.workspace(p[6], gtr_causal_conv_bwd_workspace_bytes(v.a.B, v.a.Hgrid, v.a.Wgrid, v.a.D, v.a.K), keep, bytes);
    return result(gtr_causal_conv_bwd(&v.a, dy.data_ptr(), ld, df, c.dense(at_or_none(g[0]), "grad_x", {v.B, v.N, v.D}, c.type, true),
                                      c.dense<float>(at_or_none(g[1]), "grad_w", {v.D, v.K}, at::kFloat, true),
                                      c.dense<float>(at_or_none(g[2]), "grad_bias", {v.D}, at::kFloat, false),
                                      c.dense(at_or_none(g[3]), "grad_init_state", st, c.type, false), ws, bytes, c.stream()),
                  {&g[0], &g[1], &g[2], &g[3]});
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ selective scan
struct Scan {
    const Tensor &u, &dt, &A, &Bm, &Cm;
    const Tensor *D, *z, *bias, *init;
    Call c;
    int64_t B, N, C, S;
    gtr_ssm_t a{};

    Scan(PyObject *u_, PyObject *dt_, PyObject *A_, PyObject *B_, PyObject *C_, PyObject *D_, PyObject *z_, PyObject *bias_,
         PyObject *init_, PyObject *H, PyObject *W, PyObject *dir, PyObject *softplus)
        : u(tensor(u_, "u")), dt(tensor(dt_, "dt")), A(tensor(A_, "A")), Bm(tensor(B_, "Bm")), Cm(tensor(C_, "Cm")),
          D(tensor_or_none(D_, "D")), z(tensor_or_none(z_, "z")), bias(tensor_or_none(bias_, "dt_bias")),
          init(tensor_or_none(init_, "init_state")), c(u, "u") {
        if (u.dim() != 3) refuse("u must be [B, N, channels]");
        if (A.dim() != 2) refuse("A must be [D, S]");
        B = u.size(0), N = u.size(1), C = u.size(2), S = A.size(1);
        const int h = small(H, "Hgrid"), v = small(W, "Wgrid");
        if (N != (int64_t)h * v) refuse("N=" + std::to_string(N) + " does not match the grid " + std::to_string(h) + "x" + std::to_string(v));
        if (B > 0x7fffffff || C > 0x7fffffff || S > 0x7fffffff) refuse("u is too large");
        a.B = (int)B, a.Hgrid = h, a.Wgrid = v, a.D = (int)C, a.S = (int)S;
        a.direction = small(dir, "direction");
        a.dtype = c.dtype;
        a.dt_softplus = truth(softplus);
        a.ldu = c.rows(u, "u", B, N, C);
        a.lddt = c.rows(dt, "dt", B, N, C);
        a.ldb = c.rows(Bm, "Bm", B, N, S);
        a.ldc = c.rows(Cm, "Cm", B, N, S);
        a.ldz = z ? c.rows(*z, "z", B, N, C) : 0;
        a.u = u.data_ptr(), a.dt = dt.data_ptr(), a.Bm = Bm.data_ptr(), a.Cm = Cm.data_ptr();
        a.z = z ? z->data_ptr() : nullptr;
        a.A = c.dense<float>(&A, "A", {C, S}, at::kFloat, true);
        a.Dskip = c.dense<float>(D, "D", {C}, at::kFloat, false);
        a.dt_bias = c.dense<float>(bias, "dt_bias", {C}, at::kFloat, false);
        a.init_state = c.dense<float>(init, "init_state", {B, C, S}, at::kFloat, false);
    }
};

// u, dt, A, Bm, Cm, D, z, dt_bias, init_state, out (or None), final_state (or True, None), workspace,
// Hgrid, Wgrid, direction, dt_softplus
PyObject *scan_fwd(PyObject *, PyObject *const *p, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 16);
    const Scan v(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[12], p[13], p[14], p[15]);
    const Call &c = v.c;
    const Tensor out = output(p[9] == Py_None ? Py_True : p[9], c, {v.B, v.N, v.C}, c.type, "out");
    const Tensor fin = output(p[10], c, {v.B, v.C, v.S}, at::kFloat, "final_state");
    Tensor keep;
    size_t bytes;
    void *ws = c.workspace(p[11], gtr_ssm_scan_fwd_workspace_bytes(v.a.B, v.a.Hgrid, v.a.Wgrid, v.a.D, v.a.S), keep, bytes);
    return result(gtr_ssm_scan_fwd(&v.a, c.dense(&out, "out", {v.B, v.N, v.C}, c.type, true),
                                   c.dense<float>(at_or_none(fin), "final_state", {v.B, v.C, v.S}, at::kFloat, false), ws,
                                   bytes, c.stream()),
                  {&out, &fin});
    END_HANDLE_TH_ERRORS
}

// u, dt, A, Bm, Cm, d_out, D, z, dt_bias, init_state, d_final_state, workspace, grads, want_init_grad,
// Hgrid, Wgrid, direction, dt_softplus
PyObject *scan_bwd(PyObject *, PyObject *const *p, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 18);
    const Scan v(p[0], p[1], p[2], p[3], p[4], p[6], p[7], p[8], p[9], p[14], p[15], p[16], p[17]);
    const Call &c = v.c;
    const Tensor &dy = tensor(p[5], "d_out");
    const long long ld = c.rows(dy, "d_out", v.B, v.N, v.C);
    const int64_t B = v.B, N = v.N, C = v.C, S = v.S;
    const float *df = c.dense<float>(tensor_or_none(p[10], "d_final_state"), "d_final_state", {B, C, S}, at::kFloat, false);
    std::vector<Tensor> g = given(p[12], 9);
    if (g.empty())
        g = {c.make({B, N, C}, c.type), c.make({B, N, C}, c.type), c.make({C, S}, at::kFloat), c.make({B, N, S}, c.type),
             c.make({B, N, S}, c.type), v.D ? c.make({C}, at::kFloat) : Tensor(), v.z ? c.make({B, N, C}, c.type) : Tensor(),
             v.bias ? c.make({C}, at::kFloat) : Tensor(), truth(p[13]) ? c.make({B, C, S}, at::kFloat) : Tensor()};
    if (!v.z && g[6].defined()) refuse("grad_z without z");
    gtr_ssm_grads_t o{};
    o.u = c.dense(at_or_none(g[0]), "grad_u", {B, N, C}, c.type, true);
    o.dt = c.dense(at_or_none(g[1]), "grad_dt", {B, N, C}, c.type, true);
    o.A = c.dense<float>(at_or_none(g[2]), "grad_A", {C, S}, at::kFloat, true);
    o.Bm = c.dense(at_or_none(g[3]), "grad_Bm", {B, N, S}, c.type, true);
    o.Cm = c.dense(at_or_none(g[4]), "grad_Cm", {B, N, S}, c.type, true);
    o.Dskip = c.dense<float>(at_or_none(g[5]), "grad_D", {C}, at::kFloat, false);
    o.z = c.dense(at_or_none(g[6]), "grad_z", {B, N, C}, c.type, v.z != nullptr);
    o.dt_bias = c.dense<float>(at_or_none(g[7]), "grad_dt_bias", {C}, at::kFloat, false);
    o.init_state = c.dense<float>(at_or_none(g[8]), "grad_init_state", {B, C, S}, at::kFloat, false);
    Tensor keep;
    size_t bytes;
    void *ws = c.workspace(p[11], gtr_ssm_scan_bwd_workspace_bytes(v.a.B, v.a.Hgrid, v.a.Wgrid, v.a.D, v.a.S), keep, bytes);
    return result(gtr_ssm_scan_bwd(&v.a, dy.data_ptr(), ld, df, &o, ws, bytes, c.stream()),
                  {&g[0], &g[1], &g[2], &g[3], &g[4], &g[5], &g[6], &g[7], &g[8]});
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ group norm
struct Norm {
    const Tensor &x;
    Call c;
    int64_t B, N, C, G;
    const float *gamma, *beta;
    bool has_gamma, has_beta;

    Norm(PyObject *x_, PyObject *gamma_, PyObject *beta_, PyObject *groups) : x(tensor(x_, "x")), c(x, "x") {
        if (x.dim() < 2) refuse("x must be [B, ..., C]");
        if (!x.is_contiguous()) refuse("x must be contiguous");
        B = x.size(0), C = x.size(-1), N = 1;
        for (int64_t i = 1; i + 1 < x.dim(); ++i) N *= x.size(i);
        G = integer(groups);
        if (G <= 0 || C == 0 || C % G) refuse(std::to_string(G) + " groups do not divide " + std::to_string(C) + " channels");
        if (B > 0x7fffffff || N > 0x7fffffff || C > 0x7fffffff) refuse("x is too large");
        has_gamma = gamma_ != Py_None, has_beta = beta_ != Py_None;
        gamma = c.dense<float>(tensor_or_none(gamma_, "gamma"), "gamma", {C}, at::kFloat, false);
        beta = c.dense<float>(tensor_or_none(beta_, "beta"), "beta", {C}, at::kFloat, false);
    }
};

// x, gamma, beta, out (or None), stats (or None), workspace, groups, eps, activation
PyObject *norm_fwd(PyObject *, PyObject *const *p, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 9);
    const Norm v(p[0], p[1], p[2], p[6]);
    const Call &c = v.c;
    const double eps = PyFloat_AsDouble(p[7]);
    if (eps == -1.0 && PyErr_Occurred()) throw python_error();
    const Tensor out = output(p[3] == Py_None ? Py_True : p[3], c, v.x.sizes(), c.type, "out");
    const Tensor st = output(p[4] == Py_None ? Py_True : p[4], c, {v.B, v.G, 2}, at::kFloat, "stats");
    Tensor keep;
    size_t bytes;
    void *ws = c.workspace(p[5], gtr_group_norm_fwd_workspace_bytes((int)v.B, (int)v.N, (int)v.C, (int)v.G), keep, bytes);
    return result(gtr_group_norm_fwd(v.x.data_ptr(), v.gamma, v.beta, (int)v.B, (int)v.N, (int)v.C, (int)v.G, (float)eps, c.dtype,
                                     small(p[8], "activation"), c.dense(&out, "out", v.x.sizes(), c.type, true),
                                     c.dense<float>(&st, "stats", {v.B, v.G, 2}, at::kFloat, true), ws, bytes, c.stream()),
                  {&out, &st});
    END_HANDLE_TH_ERRORS
}

// x, d_out, stats, gamma, beta, workspace, grads, groups, activation
PyObject *norm_bwd(PyObject *, PyObject *const *p, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 9);
    const Norm v(p[0], p[3], p[4], p[7]);
    const Call &c = v.c;
    const Tensor &dy = tensor(p[1], "d_out"), &st = tensor(p[2], "stats");
    const void *d = c.dense(&dy, "d_out", v.x.sizes(), c.type, true);
    const float *s = c.dense<float>(&st, "stats", {v.B, v.G, 2}, at::kFloat, true);
    std::vector<Tensor> g = given(p[6], 3);
    if (g.empty())
        g = {c.make(v.x.sizes(), c.type), v.has_gamma ? c.make({v.C}, at::kFloat) : Tensor(),
             v.has_beta ? c.make({v.C}, at::kFloat) : Tensor()};
    Tensor keep;
    size_t bytes;
    void *ws = c.workspace(p[5], gtr_group_norm_bwd_workspace_bytes((int)v.B, (int)v.N, (int)v.C, (int)v.G), keep, bytes);
    return result(gtr_group_norm_bwd(v.x.data_ptr(), d, s, v.gamma, v.beta, (int)v.B, (int)v.N, (int)v.C, (int)v.G, c.dtype,
                                     small(p[8], "activation"), c.dense(at_or_none(g[0]), "grad_x", v.x.sizes(), c.type, true),
                                     c.dense<float>(at_or_none(g[1]), "grad_gamma", {v.C}, at::kFloat, false),
                                     c.dense<float>(at_or_none(g[2]), "grad_beta", {v.C}, at::kFloat, false), ws, bytes,
                                     c.stream()),
                  {&g[0], &g[1], &g[2]});
    END_HANDLE_TH_ERRORS
}

#define GTR_ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {GTR_ENTRY(conv_fwd), GTR_ENTRY(conv_bwd), GTR_ENTRY(scan_fwd), GTR_ENTRY(scan_bwd),
                          GTR_ENTRY(norm_fwd), GTR_ENTRY(norm_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&kModule); }
