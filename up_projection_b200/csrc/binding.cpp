// binding.cpp -- the usual call of the operators around the projection without
// the interpreter's share: checks, outputs and the call of the C entry in one
// native function.  It knows the calls that are in order (plain CUDA tensors
// on the current device, of the documented types, shapes and layouts) and
// returns None for every other, which _capi.py then checks, explains or
// carries out; an int is the status of a C entry that refused.  A block norm
// of a few rows takes the host 10.6 us through ctypes and torch's Python
// functions and 4.2 us here, its backward 22.7 and 9.4, a product 10.0 and 4.1.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "swiglu.h"

namespace {

using at::Tensor;

// The C entries, from the library that _capi.py has loaded.
struct Entries {
    decltype(&swiglu_block_norm) norm;
    decltype(&swiglu_block_norm_bwd_workspace) norm_workspace;
    decltype(&swiglu_block_norm_bwd) norm_bwd;
    decltype(&swiglu_quant_b128) quant;
    decltype(&swiglu_gemm_b128) gemm;
    decltype(&swiglu_fwd_b128) fwd;
} g;

// A plain tensor (no subclass), or null.
const Tensor *plain(PyObject *o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool fits(const Tensor *t, int device, at::ScalarType dtype, at::IntArrayRef sizes) {
    return t && t->is_cuda() && t->get_device() == device && t->scalar_type() == dtype && t->sizes() == sizes &&
           t->is_contiguous();
}

bool codes(const Tensor *t, int device) {
    return t && t->is_cuda() && t->get_device() == device && t->is_contiguous() &&
           (t->scalar_type() == at::kByte || t->scalar_type() == at::kFloat8_e4m3fn);
}

int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }

// The 1 x 128 scales [rows, kb], stored [kb, rows padded to 4].
bool row_scales(const Tensor *t, int device, int64_t rows, int64_t kb) {
    return t && t->is_cuda() && t->get_device() == device && t->scalar_type() == at::kFloat && t->dim() == 2 &&
           t->size(0) == rows && t->size(1) == kb && (rows <= 1 || t->stride(0) == 1) &&
           (kb <= 1 || t->stride(1) == up4(rows));
}

Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype, int device) {
    return at::detail::empty_cuda(sizes, dtype, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)),
                                  std::nullopt);
}

void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

PyObject *wrap(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *tuple(std::initializer_list<const Tensor *> ts) {
    PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor *t : ts) {
        PyObject *o = wrap(*t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Calls a C entry without the interpreter's lock (a launch waits when the
// device's queue is full).
template <typename F>
int call(F &&f) {
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = f();
    Py_END_ALLOW_THREADS;
    return st;
}

// Runs a body that may throw (the allocator's out-of-memory error).
template <typename F>
PyObject *guarded(F &&f) {
    try {
        return f();
    } catch (const std::exception &) {
        PyErr_Clear();
        Py_RETURN_NONE;   // the caller's own path raises it as torch does
    }
}

struct Norm {
    const Tensor *y;
    int device, code;
    at::ScalarType dtype;
    int64_t M, D;
    swiglu_block_norm_params p;
    const Tensor *post = nullptr, *pre = nullptr, *gate = nullptr;

    bool read(PyObject *oy, PyObject *opost, PyObject *opre, PyObject *ogate, double scale, double eps) {
        y = plain(oy);
        if (!y || !y->is_cuda() || y->dim() < 1 || !y->is_contiguous()) return false;
        device = y->get_device();
        dtype = y->scalar_type();
        D = y->size(-1);
        if (device != c10::cuda::current_device() || (dtype != at::kBFloat16 && dtype != at::kFloat) || D == 0)
            return false;
        M = y->numel() / D;
        if (M == 0) return false;
        code = dtype == at::kFloat ? SWIGLU_FP32 : SWIGLU_BF16;
        if (opost != Py_None && !fits(post = plain(opost), device, dtype, {D})) return false;
        if (opre != Py_None && !fits(pre = plain(opre), device, dtype, {D})) return false;
        int64_t rows = 1;
        if (ogate != Py_None) {
            gate = plain(ogate);
            if (!gate) return false;
            if (gate->dim() == 2) rows = gate->size(0);
            if (rows == 0) return false;   // (its null address would read as no gate)
            if (gate->dim() == 2 ? !fits(gate, device, dtype, {rows, D}) : !fits(gate, device, dtype, {D}))
                return false;
        }
        p = {};
        p.post_weight = ptr(post);
        p.pre_weight = ptr(pre);
        p.gate = ptr(gate);
        p.gate_rows = rows;
        p.residual_scale = static_cast<float>(scale);
        p.eps = static_cast<float>(eps);
        return true;
    }
};

bool number(PyObject *o, double &v) {
    if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o)) return false;
    v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}

// (Y, R, post, pre, gate, residual_scale, eps, return_stats, Rn)
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        double scale, eps;
        Norm x;
        if (!number(a[5], scale) || !number(a[6], eps) || !x.read(a[0], a[2], a[3], a[4], scale, eps)) Py_RETURN_NONE;
        const Tensor *r = plain(a[1]), *given = a[8] != Py_None ? plain(a[8]) : nullptr;
        if (!fits(r, x.device, x.dtype, x.y->sizes()) ||
            (a[8] != Py_None && !fits(given, x.device, x.dtype, x.y->sizes())))
            Py_RETURN_NONE;
        const bool stats = a[7] == Py_True;
        if (!stats && a[7] != Py_False) Py_RETURN_NONE;
        Tensor rn = given ? *given : empty(x.y->sizes(), x.dtype, x.device), nn, r1, r2;
        if (x.pre) nn = empty(x.y->sizes(), x.dtype, x.device);
        if (stats && x.post) r1 = empty({x.M}, at::kFloat, x.device);
        if (stats && x.pre) r2 = empty({x.M}, at::kFloat, x.device);
        const cudaStream_t s = c10::cuda::getCurrentCUDAStream().stream();
        const int st = call([&] {
            return g.norm(x.y->data_ptr(), r->data_ptr(), &x.p, rn.data_ptr(), nn.defined() ? nn.data_ptr() : nullptr,
                          r1.defined() ? r1.data_ptr<float>() : nullptr, r2.defined() ? r2.data_ptr<float>() : nullptr,
                          x.M, x.D, x.code, s);
        });
        if (st) return PyLong_FromLong(st);
        return stats ? tuple({&rn, &nn, &r1, &r2}) : tuple({&rn, &nn});
    });
}

// (dRn, dN, Y, Rn, rstd_post, rstd_pre, post, pre, gate, residual_scale)
PyObject *block_norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        double scale;
        Norm x;
        if (!number(a[9], scale) || !x.read(a[2], a[6], a[7], a[8], scale, 0.0)) Py_RETURN_NONE;
        const at::IntArrayRef sizes = x.y->sizes();
        const Tensor *rn = plain(a[3]), *drn = nullptr, *dn = nullptr, *r1 = nullptr, *r2 = nullptr;
        if (!fits(rn, x.device, x.dtype, sizes) || (a[1] == Py_None) != (x.pre == nullptr)) Py_RETURN_NONE;
        if (a[0] != Py_None && !fits(drn = plain(a[0]), x.device, x.dtype, sizes)) Py_RETURN_NONE;
        if (a[1] != Py_None && !fits(dn = plain(a[1]), x.device, x.dtype, sizes)) Py_RETURN_NONE;
        if (x.post && !fits(r1 = plain(a[4]), x.device, at::kFloat, {x.M})) Py_RETURN_NONE;
        if (x.pre && !fits(r2 = plain(a[5]), x.device, at::kFloat, {x.M})) Py_RETURN_NONE;
        const int64_t need = g.norm_workspace(&x.p, x.M, x.D, x.code);
        if (need < 0) Py_RETURN_NONE;
        Tensor dy = empty(sizes, x.dtype, x.device), dr = empty(sizes, x.dtype, x.device), d1, d2, dg, ws;
        if (x.post) d1 = empty({x.D}, x.dtype, x.device);
        if (x.pre) d2 = empty({x.D}, x.dtype, x.device);
        if (x.gate) dg = empty(x.gate->sizes(), x.dtype, x.device);
        if (need > 0) ws = empty({need}, at::kByte, x.device);
        auto at_ = [](const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
        const cudaStream_t s = c10::cuda::getCurrentCUDAStream().stream();
        const int st = call([&] {
            return g.norm_bwd(ptr(drn), ptr(dn), x.y->data_ptr(), rn->data_ptr(), static_cast<const float *>(ptr(r1)),
                              static_cast<const float *>(ptr(r2)), &x.p, dy.data_ptr(), dr.data_ptr(), at_(d1), at_(d2),
                              at_(dg), at_(ws), need, x.M, x.D, x.code, s);
        });
        if (st) return PyLong_FromLong(st);
        return tuple({&dy, &dr, &d1, &d2, &dg});
    });
}

// (X, tile, transpose)
PyObject *quant_b128(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 3) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const Tensor *x = plain(a[0]);
        if (!x || !x->is_cuda() || x->dim() < 1 || !x->is_contiguous() || x->numel() == 0) Py_RETURN_NONE;
        const int device = x->get_device();
        const at::ScalarType dtype = x->scalar_type();
        if (device != c10::cuda::current_device() || (dtype != at::kBFloat16 && dtype != at::kFloat)) Py_RETURN_NONE;
        const bool tile = a[1] == Py_True, trans = a[2] == Py_True;
        if ((!tile && a[1] != Py_False) || (!trans && a[2] != Py_False)) Py_RETURN_NONE;
        const int64_t C = x->size(-1), R = x->numel() / C;
        const int64_t rows = trans ? C : R, cols = trans ? (R + 15) / 16 * 16 : C, kb = blocks128(cols);
        Tensor q = trans ? empty({rows, cols}, at::kByte, device) : empty(x->sizes(), at::kByte, device);
        Tensor s = tile ? empty({blocks128(rows), kb}, at::kFloat, device) : empty({kb, up4(rows)}, at::kFloat, device);
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream().stream();
        const int st = call([&] {
            return g.quant(x->data_ptr(), q.data_ptr(), s.data_ptr<float>(), R, C,
                           dtype == at::kFloat ? SWIGLU_FP32 : SWIGLU_BF16, tile ? SWIGLU_BLOCK_TILE : SWIGLU_BLOCK_ROW,
                           trans ? 1 : 0, stream);
        });
        if (st) return PyLong_FromLong(st);
        // (row scales: the rows innermost; the tensor is this call's own)
        if (!tile) {
            const int64_t sizes[2] = {rows, kb}, strides[2] = {1, up4(rows)};
            s.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(sizes, 2), at::IntArrayRef(strides, 2));
        }
        return tuple({&q, &s});
    });
}

// (A, As, B, Bs, fp32 result, Y)
PyObject *gemm_b128(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const Tensor *A = plain(a[0]), *As = plain(a[1]), *B = plain(a[2]), *Bs = plain(a[3]);
        const int device = c10::cuda::current_device();
        if (!codes(A, device) || !codes(B, device) || A->dim() < 1 || B->dim() != 2 || A->numel() == 0) Py_RETURN_NONE;
        const int64_t K = A->size(-1), M = A->numel() / K, N = B->size(0), kb = blocks128(K);
        if (B->size(1) != K || !row_scales(As, device, M, kb)) Py_RETURN_NONE;
        const bool tile = fits(Bs, device, at::kFloat, {blocks128(N), kb});
        if (!tile && !row_scales(Bs, device, N, kb)) Py_RETURN_NONE;
        const bool f32 = a[4] == Py_True;
        const at::ScalarType dtype = f32 ? at::kFloat : at::kBFloat16;
        Tensor y;
        if (a[5] != Py_None) {
            const Tensor *given = plain(a[5]);
            if (!given || !given->is_cuda() || given->get_device() != device || !given->is_contiguous() ||
                given->scalar_type() != dtype || given->numel() != M * N)
                Py_RETURN_NONE;
            y = *given;
        } else {
            at::DimVector sizes(A->sizes());
            sizes.back() = N;
            y = empty(sizes, dtype, device);
        }
        const cudaStream_t s = c10::cuda::getCurrentCUDAStream().stream();
        const int st = call([&] {
            return g.gemm(A->data_ptr(), As->data_ptr<float>(), B->data_ptr(), Bs->data_ptr<float>(), y.data_ptr(), M, N,
                          K, tile ? SWIGLU_BLOCK_TILE : SWIGLU_BLOCK_ROW, f32 ? SWIGLU_FP32 : SWIGLU_BF16, s);
        });
        if (st) return PyLong_FromLong(st);
        return wrap(y);
    });
}

// (X, Xs, Wg, Wgs, Wu, Wus, H, activation, gate_multiplier, return_gu)
PyObject *fwd_b128(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const Tensor *X = plain(a[0]), *Xs = plain(a[1]), *Wg = plain(a[2]), *Wgs = plain(a[3]), *Wu = plain(a[4]),
                     *Wus = plain(a[5]);
        const int device = c10::cuda::current_device();
        if (!codes(X, device) || !codes(Wg, device) || !codes(Wu, device) || X->dim() < 1 || Wg->dim() != 2 ||
            X->numel() == 0)
            Py_RETURN_NONE;
        const int64_t K = X->size(-1), M = X->numel() / K, N = Wg->size(0), kb = blocks128(K), nb = blocks128(N);
        if (Wg->size(1) != K || Wu->sizes() != Wg->sizes() || !row_scales(Xs, device, M, kb) ||
            !fits(Wgs, device, at::kFloat, {nb, kb}) || !fits(Wus, device, at::kFloat, {nb, kb}))
            Py_RETURN_NONE;
        double alpha;
        const long act = PyLong_CheckExact(a[7]) ? PyLong_AsLong(a[7]) : -1;
        const bool gu = a[9] == Py_True;
        if (PyErr_Occurred() || !number(a[8], alpha) || act < 0 || act > INT_MAX || (!gu && a[9] != Py_False)) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        Tensor h, G, U;
        if (a[6] != Py_None) {
            const Tensor *given = plain(a[6]);
            if (!given || !given->is_cuda() || given->get_device() != device || !given->is_contiguous() ||
                given->scalar_type() != at::kBFloat16 || given->numel() != M * N)
                Py_RETURN_NONE;
            h = *given;
        } else {
            at::DimVector sizes(X->sizes());
            sizes.back() = N;
            h = empty(sizes, at::kBFloat16, device);
        }
        swiglu_epilogue epi = {};
        epi.activation = static_cast<int>(act);
        epi.gate_multiplier = static_cast<float>(alpha);
        if (gu) {
            G = empty(h.sizes(), at::kBFloat16, device);
            U = empty(h.sizes(), at::kBFloat16, device);
            epi.G = G.data_ptr();
            epi.U = U.data_ptr();
        }
        const cudaStream_t s = c10::cuda::getCurrentCUDAStream().stream();
        const int st = call([&] {
            return g.fwd(X->data_ptr(), Xs->data_ptr<float>(), Wg->data_ptr(), Wgs->data_ptr<float>(), Wu->data_ptr(),
                         Wus->data_ptr<float>(), h.data_ptr(), M, K, N, &epi, s);
        });
        if (st) return PyLong_FromLong(st);
        return gu ? tuple({&h, &G, &U}) : wrap(h);
    });
}

// Addresses of the C entries, in the order of Entries.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "six addresses");
        return nullptr;
    }
    void *p[6];
    for (int i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    g.norm = reinterpret_cast<decltype(g.norm)>(p[0]);
    g.norm_workspace = reinterpret_cast<decltype(g.norm_workspace)>(p[1]);
    g.norm_bwd = reinterpret_cast<decltype(g.norm_bwd)>(p[2]);
    g.quant = reinterpret_cast<decltype(g.quant)>(p[3]);
    g.gemm = reinterpret_cast<decltype(g.gemm)>(p[4]);
    g.fwd = reinterpret_cast<decltype(g.fwd)>(p[5]);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"block_norm", fast(block_norm), METH_FASTCALL, nullptr},
    {"block_norm_bwd", fast(block_norm_bwd), METH_FASTCALL, nullptr},
    {"quant_b128", fast(quant_b128), METH_FASTCALL, nullptr},
    {"gemm_b128", fast(gemm_b128), METH_FASTCALL, nullptr},
    {"fwd_b128", fast(fwd_b128), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Native calls of the operators around the projection.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (SWIGLU_BUILT_FOR: the torch, ABI and interpreter of these headers, which the
// importer compares with its own before the first call)
PyMODINIT_FUNC PyInit__binding() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", SWIGLU_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
