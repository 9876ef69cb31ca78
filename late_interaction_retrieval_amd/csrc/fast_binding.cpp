// fast_binding.cpp -- the usual calls of binding.py's embedding-head operators
// as a Python extension (_fast.so): on small tensors the interpreter's share of a
// call (6 us) was more than the kernel's.
//
// Each function takes its binding function's main arguments.  It makes the call where
// they are plain -- contiguous tensors of the right types and sizes on the
// current device, outputs to be allocated -- and returns its results; anything
// else, and any status but MAXSIM_OK, gives None, and the binding function
// goes its own way, which handles the general case and names what is wrong.
// adamw() returns the status instead, and None only where it made no call: a step
// in place that may have been launched must not be made again.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "maxsim_encoder.h"

namespace {

using at::Tensor;

int code_of(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return MAXSIM_F16;
        case at::kBFloat16: return MAXSIM_BF16;
        case at::kFloat: return MAXSIM_F32;
        case at::kChar: return MAXSIM_I8;
        case at::kFloat8_e4m3fn: return MAXSIM_E4M3;
        default: return -1;
    }
}
bool is_float(int code) { return code >= MAXSIM_F16 && code <= MAXSIM_F32; }
int64_t blocks(int64_t n) { return (n + MAXSIM_QBLOCK - 1) / MAXSIM_QBLOCK; }

// A tensor argument; nullptr for None.  `plain` turns false for anything else.
const Tensor* tensor(PyObject* o, bool& plain) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
        plain = false;
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}
// Contiguous, of this type and on this device.
bool good(const Tensor& t, at::ScalarType type, at::Device dev) {
    return t.scalar_type() == type && t.device() == dev && t.is_contiguous();
}
bool on_current(const Tensor& t) { return t.is_cuda() && t.device().index() == c10::hip::current_device(); }
void* stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }
void* at_(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
bool fits(int64_t n) { return n <= INT32_MAX; }

Tensor empty(at::IntArrayRef shape, const Tensor& like, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type).requires_grad(false));
}
int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }
// [rows, width] e4m3 in rows a multiple of 16 bytes apart, as the product reads them.
Tensor empty_e4m3(int64_t rows, int64_t width, const Tensor& like) {
    const int64_t pitch = round16(width);
    Tensor t = empty({rows, pitch}, like, at::kFloat8_e4m3fn);
    return pitch == width ? t : t.narrow(1, 0, width);
}
// The pitch of such an operand, every row of which is readable up to its width rounded up to 16; 0: not one.
int64_t operand_pitch(const Tensor& t, at::Device dev) {
    if (t.scalar_type() != at::kFloat8_e4m3fn || t.device() != dev || t.dim() != 2) return 0;
    const int64_t rows = t.size(0), width = t.size(1), wide = round16(width);
    if (wide == width && t.is_contiguous()) return width;
    if (rows < 1 || width < 1 || t.stride(1) != 1) return 0;
    const int64_t ld = rows == 1 ? wide : t.stride(0);
    if (ld < wide || t.storage_offset() + (rows - 1) * ld + wide > (int64_t)t.storage().nbytes()) return 0;
    return ld;
}
PyObject* wrap(const Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
PyObject* tuple(std::initializer_list<Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) {
        PyObject* o = wrap(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// (x, weight, eps, residual, out_dtype or None, with_rstd) -> (y, scale, sum, rstd)
PyObject* rmsnorm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool plain = n == 6 && (a[4] == Py_None || THPDtype_Check(a[4]));
    if (!plain) Py_RETURN_NONE;
    const Tensor *x = tensor(a[0], plain), *w = tensor(a[1], plain), *res = tensor(a[3], plain);
    const double eps = PyFloat_Check(a[2]) ? PyFloat_AS_DOUBLE(a[2]) : -1;
    if (!plain || !x || eps < 0 || x->dim() < 1 || !on_current(*x) || !x->is_contiguous()) Py_RETURN_NONE;
    const at::ScalarType type = x->scalar_type();
    const at::ScalarType out = a[4] == Py_None ? type : reinterpret_cast<THPDtype*>(a[4])->scalar_type;
    const int code = code_of(type), out_code = code_of(out);
    const int64_t H = x->size(-1), R = H ? x->numel() / H : 0;
    const bool odd = out_code == MAXSIM_E4M3 && H % 16 != 0;  // rows that are padded
    if (!is_float(code) || out_code < 0 || H < 1 || !fits(H) || !fits(R) || (odd && x->dim() != 2)) Py_RETURN_NONE;
    if (w && (!(good(*w, type, x->device()) || good(*w, at::kFloat, x->device())) || w->numel() != H)) Py_RETURN_NONE;
    if (res && (!good(*res, type, x->device()) || res->sizes() != x->sizes())) Py_RETURN_NONE;
    const int rstd_wanted = PyObject_IsTrue(a[5]);
    if (rstd_wanted < 0) return nullptr;
    Tensor y = odd ? empty_e4m3(R, H, *x) : empty(x->sizes(), *x, out), scale, sum, rstd;
    const at::IntArrayRef rows = x->sizes().slice(0, x->dim() - 1);
    if (out_code == MAXSIM_I8) scale = empty(rows, *x, at::kFloat);
    if (out_code == MAXSIM_E4M3) {
        std::vector<int64_t> shape = rows.vec();
        shape.push_back(blocks(H));
        scale = empty(shape, *x, at::kFloat);
    }
    if (res) sum = empty(x->sizes(), *x, type);
    if (rstd_wanted) rstd = empty(rows, *x, at::kFloat);
    if (maxsim_rmsnorm_fwd(x->data_ptr(), H, at_(res), H, at_(w), w ? code_of(w->scalar_type()) : MAXSIM_F32, (int32_t)R,
                           (int32_t)H, code, (float)eps, out_code, y.data_ptr(), odd ? round16(H) : H,
                           scale.defined() ? scale.data_ptr<float>() : nullptr, sum.defined() ? sum.data_ptr() : nullptr,
                           H, rstd.defined() ? rstd.data_ptr<float>() : nullptr, stream_of(*x)) != MAXSIM_OK)
        Py_RETURN_NONE;
    return tuple({y, scale, sum, rstd});
    END_HANDLE_TH_ERRORS
}

// (dy, h, rstd, weight, dsum, with_dweight) -> (dx, dweight)
PyObject* rmsnorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool plain = n == 6;
    if (!plain) Py_RETURN_NONE;
    const Tensor *dy = tensor(a[0], plain), *h = tensor(a[1], plain), *rstd = tensor(a[2], plain),
                 *w = tensor(a[3], plain), *ds = tensor(a[4], plain);
    if (!plain || !dy || !h || !rstd || h->dim() < 1 || !on_current(*h) || !h->is_contiguous()) Py_RETURN_NONE;
    const at::ScalarType type = h->scalar_type();
    const int code = code_of(type);
    const int64_t H = h->size(-1), R = H ? h->numel() / H : 0;
    if (!is_float(code) || H < 1 || !fits(H) || !fits(R)) Py_RETURN_NONE;
    if (!good(*dy, type, h->device()) || dy->sizes() != h->sizes() || !good(*rstd, at::kFloat, h->device()) ||
        rstd->numel() != R)
        Py_RETURN_NONE;
    if (w && (!(good(*w, type, h->device()) || good(*w, at::kFloat, h->device())) || w->numel() != H)) Py_RETURN_NONE;
    if (ds && (!good(*ds, type, h->device()) || ds->sizes() != h->sizes())) Py_RETURN_NONE;
    const int dw_wanted = PyObject_IsTrue(a[5]);
    if (dw_wanted < 0) return nullptr;
    Tensor dx = empty(h->sizes(), *h, type), dw, ws;
    size_t bytes = 0;
    if (dw_wanted) {
        dw = empty({H}, *h, at::kFloat);
        bytes = maxsim_rmsnorm_bwd_workspace_bytes((int32_t)R, (int32_t)H);
        if (bytes) ws = empty({(int64_t)bytes}, *h, at::kByte);
    }
    if (maxsim_rmsnorm_bwd(dy->data_ptr(), H, h->data_ptr(), H, rstd->data_ptr<float>(), at_(w),
                           w ? code_of(w->scalar_type()) : MAXSIM_F32, at_(ds), H, (int32_t)R, (int32_t)H, code,
                           dx.data_ptr(), H, dw_wanted ? dw.data_ptr<float>() : nullptr,
                           bytes ? ws.data_ptr() : nullptr, bytes, stream_of(*h)) != MAXSIM_OK)
        Py_RETURN_NONE;
    return tuple({dx, dw});
    END_HANDLE_TH_ERRORS
}

// (x, block_rows, rows, transposed) -> (q, scale, qt, scale_t)
PyObject* quant_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool plain = n == 4;
    if (!plain) Py_RETURN_NONE;
    const Tensor* x = tensor(a[0], plain);
    const long br = PyLong_Check(a[1]) ? PyLong_AsLong(a[1]) : 0;
    if (br == -1 && PyErr_Occurred()) PyErr_Clear();
    const int rows = PyObject_IsTrue(a[2]), both = PyObject_IsTrue(a[3]);
    if (rows < 0 || both < 0) return nullptr;
    if (!plain || !x || x->dim() != 2 || !on_current(*x) || !x->is_contiguous() || (br != 1 && br != MAXSIM_QBLOCK) ||
        (!rows && !both))
        Py_RETURN_NONE;
    const int code = code_of(x->scalar_type());
    const int64_t R = x->size(0), C = x->size(1);
    if (!is_float(code) || !fits(R) || !fits(C)) Py_RETURN_NONE;
    Tensor q, scale, qt, scale_t;
    if (rows) {
        q = empty_e4m3(R, C, *x);
        scale = empty({br == 1 ? R : blocks(R), blocks(C)}, *x, at::kFloat);
    }
    if (both) {
        qt = empty_e4m3(C, R, *x);
        scale_t = empty({br == 1 ? C : blocks(C), blocks(R)}, *x, at::kFloat);
    }
    if (maxsim_quant_fp8(x->data_ptr(), C, (int32_t)R, (int32_t)C, code, (int32_t)br, rows ? q.data_ptr() : nullptr,
                         round16(C),
                         rows ? scale.data_ptr<float>() : nullptr, both ? qt.data_ptr() : nullptr, round16(R),
                         both ? scale_t.data_ptr<float>() : nullptr, stream_of(*x)) != MAXSIM_OK)
        Py_RETURN_NONE;
    return tuple({q, scale, qt, scale_t});
    END_HANDLE_TH_ERRORS
}

// (A, a_scale, B, b_scale, out_dtype) -> c
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool plain = n == 5 && THPDtype_Check(a[4]);
    if (!plain) Py_RETURN_NONE;
    const Tensor *A = tensor(a[0], plain), *sa = tensor(a[1], plain), *B = tensor(a[2], plain), *sb = tensor(a[3], plain);
    if (!plain || !A || !sa || !B || !sb || A->dim() != 2 || B->dim() != 2 || sb->dim() != 2 || !on_current(*A))
        Py_RETURN_NONE;
    const at::Device dev = A->device();
    const int64_t M = A->size(0), K = A->size(1), N = B->size(0), kb = blocks(K);
    const at::ScalarType out = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
    const int64_t lda = operand_pitch(*A, dev), ldb = operand_pitch(*B, dev);
    if (!lda || !ldb || !good(*sa, at::kFloat, dev) || !good(*sb, at::kFloat, dev) || B->size(1) != K || !fits(M) ||
        !fits(N) || !fits(K) || !is_float(code_of(out)))
        Py_RETURN_NONE;
    const int32_t rows = sb->size(0) == N ? 1 : MAXSIM_QBLOCK;
    if (sa->numel() != M * kb || sb->numel() != (rows == 1 ? N : blocks(N)) * kb) Py_RETURN_NONE;
    Tensor c = empty({M, N}, *A, out), ws;
    const size_t bytes = maxsim_gemm_fp8_workspace_bytes((int32_t)M, (int32_t)N, (int32_t)K);
    if (bytes) ws = empty({(int64_t)bytes}, *A, at::kByte);
    if (maxsim_gemm_fp8(A->data_ptr(), lda, sa->data_ptr<float>(), B->data_ptr(), ldb, sb->data_ptr<float>(), rows, (int32_t)M,
                        (int32_t)N, (int32_t)K, code_of(out), c.data_ptr(), N, bytes ? ws.data_ptr() : nullptr, bytes,
                        stream_of(*A)) != MAXSIM_OK)
        Py_RETURN_NONE;
    return wrap(c);
    END_HANDLE_TH_ERRORS
}

// (table address, count, device index, param code, state code, held, grads, lr, beta1, beta2, eps, decay, step) ->
// the call's status: the table's entries with these gradients; its own memory is not written.  held: for each entry the tensors
// param, m, v, (with 8-bit states) m_scale, v_scale, (with masters) master, which must be where the table says.
PyObject* adamw(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 13 || !PyList_Check(a[5]) || !PyList_Check(a[6])) Py_RETURN_NONE;
    const auto* table = reinterpret_cast<const maxsim_adamw_tensor*>(PyLong_AsVoidPtr(a[0]));
    const Py_ssize_t count = PyLong_AsSsize_t(a[1]);
    const long device = PyLong_AsLong(a[2]), param = PyLong_AsLong(a[3]), state = PyLong_AsLong(a[4]);
    double v[5];
    for (int i = 0; i < 5; ++i) v[i] = PyFloat_AsDouble(a[7 + i]);
    const long step = PyLong_AsLong(a[12]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (count < 1 || PyList_GET_SIZE(a[6]) != count || step < 1 || step > INT32_MAX ||
        device != c10::hip::current_device())
        Py_RETURN_NONE;
    std::vector<maxsim_adamw_tensor> t(table, table + count);
    const bool packed = state == MAXSIM_E4M3;
    const Py_ssize_t each = PyList_GET_SIZE(a[5]) / count, states = packed ? 5 : 3;
    if (PyList_GET_SIZE(a[5]) != each * count || (each != states && each != states + 1)) Py_RETURN_NONE;
    for (Py_ssize_t i = 0; i < count; ++i) {
        const void* at[6] = {t[i].param, t[i].m, t[i].v, t[i].m_scale, t[i].v_scale, nullptr};
        at[states] = t[i].master;
        for (Py_ssize_t j = 0; j < each; ++j) {
            bool plain = true;
            const Tensor* held = tensor(PyList_GET_ITEM(a[5], i * each + j), plain);
            if (!held || held->data_ptr() != at[j]) Py_RETURN_NONE;
        }
    }
    at::ScalarType type = at::kFloat;
    for (Py_ssize_t i = 0; i < count; ++i) {
        bool plain = true;
        const Tensor* g = tensor(PyList_GET_ITEM(a[6], i), plain);
        if (!g || !g->is_cuda() || g->device().index() != device || !g->is_contiguous() || g->numel() != t[i].n)
            Py_RETURN_NONE;
        if (i == 0) type = g->scalar_type();
        if (g->scalar_type() != type) Py_RETURN_NONE;
        t[i].grad = g->data_ptr();
    }
    void* stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
    if (!is_float(code_of(type))) Py_RETURN_NONE;
    const int status = maxsim_adamw(t.data(), (int32_t)count, (int32_t)param, code_of(type), (int32_t)state, v[0], v[1], v[2],
                                    v[3], v[4], (int32_t)step, nullptr, stream);
    if (status == MAXSIM_OK || status == MAXSIM_ERR_HIP) {  // the parameters have changed, or some may have
        for (Py_ssize_t i = 0; i < count; ++i) {
            const Tensor& param = THPVariable_Unpack(PyList_GET_ITEM(a[5], i * each));
            if (!param.is_inference()) param.unsafeGetTensorImpl()->bump_version();
        }
    }
    return PyLong_FromLong(status);
    END_HANDLE_TH_ERRORS
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rmsnorm_fwd), FAST(rmsnorm_bwd), FAST(quant_fp8), FAST(gemm_fp8), FAST(adamw),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&module); }
