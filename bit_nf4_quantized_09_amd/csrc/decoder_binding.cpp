// decoder_binding.cpp -- the Python calls of the operators around the linears, over the C ABI of
// include/qlora_decoder.h.
//
// A CPython extension of its own, because a call that serves single tokens lasts as long as its host
// side: a call that turns q and k of a few tokens took 13.8 us through ctypes and takes 5.5 us here (4.3 us
// of them the launch); one that appends a token 13.5 and 6.6, one that attends from it 11.4 and 5.9.  It only
// marshals: types, shapes, strides and devices are checked, outputs and workspaces are
// allocated with torch, and raw pointers go to the library with torch's current stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "../../include/qlora_decoder.h"

namespace {

PyObject* g_error = nullptr;       // NF4Error
PyObject* g_stream = nullptr;      // torch's current stream of a device, as an integer

struct BadValue {
    std::string what;
};
struct BadType {
    std::string what;
};
struct PythonError {};             // already set

[[noreturn]] void bad(const std::string& what) { throw BadValue{what}; }

void check(nf4_status st) {
    if (st == NF4_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, nf4_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw PythonError{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw BadType{std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}
int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError{};
    return v != 0;
}

std::string shape_of(const at::Tensor& t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}
const char* type_name(at::ScalarType t) { return c10::toString(t); }

void want_type(const at::Tensor& t, const char* name, at::ScalarType type) {
    if (t.scalar_type() != type) bad(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
}
void want_gpu(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) bad(std::string(name) + " must be a GPU tensor");
}
void want_device(const at::Tensor& t, const char* name, const at::Tensor& of) {
    if (t.device() != of.device())
        bad(std::string(name) + " must be on the same GPU as the other operands (" + of.device().str() + "), got " + t.device().str());
}
// A dense operand on the device of `of`.
void want_dense(const at::Tensor& t, const char* name, at::ScalarType type, const at::Tensor& of) {
    want_type(t, name, type);
    want_device(t, name, of);
    if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
}

void* stream_of(const at::Tensor& t) {
    PyObject* index = PyLong_FromLong(t.get_device());
    if (!index) throw PythonError{};
    PyObject* s = PyObject_CallOneArg(g_stream, index);
    Py_DECREF(index);
    if (!s) throw PythonError{};
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw PythonError{};
    return p;
}

// A [tokens, heads, dim] tensor of any token and head strides.
qlora_heads heads_of(const at::Tensor& t, const char* name, at::ScalarType type, int64_t tokens, int64_t dim, const at::Tensor& of) {
    want_type(t, name, type);
    want_device(t, name, of);
    if (t.dim() != 3 || t.size(0) != tokens || t.size(2) != dim || t.size(1) < 1 || t.size(1) > 65536)
        bad(std::string(name) + " must be [" + std::to_string(tokens) + ", heads, " + std::to_string(dim) + "], got " + shape_of(t));
    if (tokens > 0 && dim > 1 && t.stride(2) != 1) bad(std::string(name) + " must be dense along its last dimension");
    const int64_t heads = t.size(1);
    const int64_t head_stride = heads > 1 ? t.stride(1) : dim;       // the stride of a dimension of one is not looked at
    return qlora_heads{t.data_ptr(), tokens > 1 ? t.stride(0) : heads * head_stride, head_stride, (int32_t)heads};
}
at::Tensor fresh_like(const at::Tensor& t, qlora_heads& h) {
    at::Tensor out = at::empty(t.sizes(), t.options());
    h = qlora_heads{out.data_ptr(), t.size(1) * t.size(2), t.size(2), (int32_t)t.size(1)};
    return out;
}

// A caller's tensor that the call has written through its pointer: its version moves on, so that autograd refuses a
// backward that saved it before (tensors of inference mode have none).
void written(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

qlora_rope rope_of(PyObject* const* a, const at::Tensor& of) {       // freq, rotary_dim, interleaved, magnitude
    const at::Tensor& freq = tensor(a[0], "freq");
    want_dense(freq, "freq", at::kLong, of);
    const int64_t rotary = whole(a[1]);
    if (rotary < 0 || rotary > 65536 || freq.numel() * 2 != rotary) bad("freq must hold rotary_dim / 2 values");
    return qlora_rope{freq.data_ptr<int64_t>(), (int32_t)rotary, truth(a[2]) ? 1 : 0, (float)number(a[3])};
}

qlora_kv_cache cache_of(PyObject* codes_o, PyObject* scales_o, const at::Tensor& of) {
    const at::Tensor &codes = tensor(codes_o, "codes"), &scales = tensor(scales_o, "scales");
    want_dense(codes, "codes", at::kByte, of);
    want_dense(scales, "scales", at::kFloat, of);
    if (codes.dim() != 5 || codes.size(1) != 2)
        bad("codes must be [pages, 2, kv_heads, page_size, head_dim], got " + shape_of(codes));
    if (scales.dim() != 3 || scales.size(0) != codes.size(0) || scales.size(1) != 2 || scales.size(2) != codes.size(2))
        bad("scales must be [pages, 2, kv_heads] as codes " + shape_of(codes) + ", got " + shape_of(scales));
    auto small = [](int64_t n) { return (int32_t)(n < 0x7FFFFFFF ? n : 0x7FFFFFFF); };
    return qlora_kv_cache{(uint8_t*)codes.data_ptr(), scales.data_ptr<float>(), codes.size(0), small(codes.size(2)),
                          small(codes.size(3)), small(codes.size(4))};
}

qlora_kv_batch batch_of(PyObject* starts_o, PyObject* lengths_o, PyObject* table_o, int64_t tokens, const at::Tensor& of) {
    const at::Tensor &starts = tensor(starts_o, "starts"), &lengths = tensor(lengths_o, "lengths"), &table = tensor(table_o, "table");
    want_dense(starts, "starts", at::kInt, of);
    want_dense(lengths, "lengths", at::kInt, of);
    want_type(table, "table", at::kInt);
    want_device(table, "table", of);
    if (table.dim() != 2) bad("table must be [seqs, pages of a sequence], got " + shape_of(table));
    const int64_t seqs = table.size(0), width = table.size(1);
    if (lengths.dim() != 1 || lengths.size(0) != seqs || starts.dim() != 1 || starts.size(0) != seqs + 1)
        bad("lengths must be [seqs] and starts [seqs + 1], as the table has " + std::to_string(seqs) + " rows");
    if (width > 1 && table.stride(1) != 1) bad("table must be dense along its rows");
    if (seqs > 0x7FFFFFFF || width > 0x7FFFFFFF) bad("table is too large");
    return qlora_kv_batch{starts.data_ptr<int32_t>(), lengths.data_ptr<int32_t>(), table.data_ptr<int32_t>(),
                          seqs > 1 ? table.stride(0) : width, tokens, (int32_t)seqs, (int32_t)width};
}

// `bytes` of workspace, 256-byte aligned (the tensor keeps it until the call has been enqueued).
void* workspace(size_t bytes, const at::Tensor& of, at::Tensor& keep) {
    if (bytes == 0) return nullptr;
    keep = at::empty({(int64_t)bytes + 256}, of.options().dtype(at::kByte));
    return (void*)(((uintptr_t)keep.data_ptr() + 255) & ~(uintptr_t)255);
}

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const BadValue& e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
    } catch (const BadType& e) {
        PyErr_SetString(PyExc_TypeError, e.what.c_str());
    } catch (const PythonError&) {
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// freq, rotary_dim, interleaved, magnitude, backward, positions, q, k or None, inplace
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const at::Tensor &positions = tensor(a[5], "positions"), &q = tensor(a[6], "q");
        want_gpu(q, "q");
        const c10::DeviceGuard on(q.device());
        const at::ScalarType type = q.scalar_type();
        if (type != at::kFloat && type != at::kBFloat16) bad(std::string("q must be Float or BFloat16, got ") + type_name(type));
        want_dense(positions, "positions", at::kInt, q);
        if (q.dim() != 3) bad("q must be [tokens, heads, dim], got " + shape_of(q));
        const int64_t M = positions.numel(), dim = q.size(2);
        if (dim > 65536) bad("q has too large heads");
        const qlora_rope r = rope_of(a, q);
        const bool two = a[7] != Py_None, inplace = truth(a[8]);
        qlora_heads in[2] = {heads_of(q, "q", type, M, dim, q)}, out[2];
        if (two) in[1] = heads_of(tensor(a[7], "k"), "k", type, M, dim, q);
        at::Tensor yq = q, yk;
        if (two) yk = tensor(a[7], "k");
        if (inplace) {
            // (autograd would not see the rotation and give the gradient of a step without it)
            if (c10::GradMode::is_enabled() && (yq.requires_grad() || (two && yk.requires_grad())))
                bad("a tensor that requires grad is not rotated in place while gradients are recorded");
            out[0] = in[0];
            out[1] = in[1];
        } else {
            yq = fresh_like(q, out[0]);
            if (two) yk = fresh_like(yk, out[1]);
        }
        check(qlora_rope_apply(&r, truth(a[4]) ? 1 : 0, (const int32_t*)positions.data_ptr(), M, (int32_t)dim,
                               type == at::kBFloat16 ? NF4_BF16 : NF4_F32, in, out, two ? 2 : 1, stream_of(q)));
        if (inplace) {
            written(yq);
            if (two) written(yk);
        }
        if (!two) return wrap(yq);
        PyObject* pq = wrap(yq);
        PyObject* pk = pq ? wrap(yk) : nullptr;
        if (!pk) {
            Py_XDECREF(pq);
            throw PythonError{};
        }
        PyObject* t = PyTuple_Pack(2, pq, pk);
        Py_DECREF(pq);
        Py_DECREF(pk);
        return t;
    });
}

// codes, scales, k, v, starts, lengths, table, q or None, then freq (or None), rotary_dim, interleaved, magnitude
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
        want_gpu(k, "k");
        const c10::DeviceGuard on(k.device());
        const qlora_kv_cache c = cache_of(a[0], a[1], k);
        const int64_t T = k.dim() > 0 ? k.size(0) : 0;
        const qlora_kv_batch b = batch_of(a[4], a[5], a[6], T, k);
        const qlora_heads kh = heads_of(k, "k", at::kBFloat16, T, c.head_dim, k), vh = heads_of(v, "v", at::kBFloat16, T, c.head_dim, k);
        qlora_rope r{};
        const bool turns = a[8] != Py_None, queries = a[7] != Py_None;
        if (turns) r = rope_of(a + 8, k);
        qlora_heads qh{}, oh{};
        at::Tensor out;
        if (queries) {
            const at::Tensor& q = tensor(a[7], "q");
            qh = heads_of(q, "q", at::kBFloat16, T, c.head_dim, k);
            out = fresh_like(q, oh);
        }
        check(qlora_kv_append(&c, &b, &kh, &vh, turns ? &r : nullptr, queries ? &qh : nullptr, queries ? &oh : nullptr, stream_of(k)));
        written(tensor(a[0], "codes"));
        written(tensor(a[1], "scales"));
        return wrap(out);
    });
}

// codes, scales, q, starts, lengths, table, scale or None, max_new or None, max_length or None
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const at::Tensor& q = tensor(a[2], "q");
        want_gpu(q, "q");
        const c10::DeviceGuard on(q.device());
        const qlora_kv_cache c = cache_of(a[0], a[1], q);
        const int64_t T = q.dim() > 0 ? q.size(0) : 0;
        const qlora_kv_batch b = batch_of(a[3], a[4], a[5], T, q);
        const qlora_heads qh = heads_of(q, "q", at::kBFloat16, T, c.head_dim, q);
        const double scale = a[6] == Py_None ? 1.0 / std::sqrt((double)c.head_dim) : number(a[6]);
        const int64_t reach = (int64_t)b.table_width * c.page_size;
        const int64_t max_new = a[7] == Py_None ? (T > 1 ? T : 1) : whole(a[7]);
        const int64_t max_length = a[8] == Py_None ? (reach > 1 ? reach : 1) : whole(a[8]);
        qlora_heads oh;
        at::Tensor out = fresh_like(q, oh), keep;
        const size_t bytes = qlora_kv_attention_workspace_bytes(&c, &b, qh.heads, max_new, max_length);
        void* ws = workspace(bytes, q, keep);
        check(qlora_kv_attention(&c, &b, &qh, &oh, (float)scale, max_new, max_length, ws, bytes, stream_of(q)));
        return wrap(out);
    });
}

// X, W, targets, dloss or None, need_dw, ignore_index
PyObject* head_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        const at::Tensor &X = tensor(a[0], "X"), &W = tensor(a[1], "W"), &targets = tensor(a[2], "targets");
        want_gpu(X, "X");
        const c10::DeviceGuard on(X.device());
        want_dense(X, "X", at::kBFloat16, X);
        want_dense(W, "W", at::kBFloat16, X);
        want_dense(targets, "targets", at::kLong, X);
        if (X.dim() != 2 || W.dim() != 2 || X.size(1) != W.size(1)) bad("X must be [M, K] and W [V, K]");
        const int64_t M = X.size(0), K = X.size(1), V = W.size(0);
        if (targets.dim() != 1 || targets.size(0) != M) bad("targets must be [" + std::to_string(M) + "]");
        const bool grad = a[3] != Py_None, dw = truth(a[4]);
        const float* dl = nullptr;
        if (grad) {
            const at::Tensor& dloss = tensor(a[3], "dloss");
            want_dense(dloss, "dloss", at::kFloat, X);
            if (dloss.dim() != 1 || dloss.size(0) != M) bad("dloss must be [" + std::to_string(M) + "]");
            dl = dloss.data_ptr<float>();
        } else if (dw) {
            bad("need_dw needs dloss");
        }
        at::Tensor loss = at::empty({M}, X.options().dtype(at::kFloat)), dX, dW, keep;
        if (grad) dX = at::empty({M, K}, X.options());
        if (dw) dW = at::empty({V, K}, X.options());
        const size_t bytes = qlora_head_loss_workspace_bytes(M, K, V, grad, dw);
        void* ws = workspace(bytes, X, keep);
        check(qlora_head_loss(X.data_ptr(), M, K, W.data_ptr(), V, targets.data_ptr<int64_t>(), whole(a[5]), dl, loss.data_ptr<float>(),
                              grad ? dX.data_ptr() : nullptr, dw ? dW.data_ptr() : nullptr, ws, bytes, stream_of(X)));
        PyObject* out[3] = {wrap(loss), wrap(dX), wrap(dW)};
        PyObject* t = out[0] && out[1] && out[2] ? PyTuple_Pack(3, out[0], out[1], out[2]) : nullptr;
        for (PyObject* o : out) Py_XDECREF(o);
        if (!t) throw PythonError{};
        return t;
    });
}

// the error class, and the function that gives a device's current stream
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 2, [&]() -> PyObject* {
        Py_INCREF(a[0]);
        Py_INCREF(a[1]);
        Py_XSETREF(g_error, a[0]);
        Py_XSETREF(g_stream, a[1]);
        Py_RETURN_NONE;
    });
}

#define CALL(f) (PyCFunction)(void*)f, METH_FASTCALL
PyMethodDef methods[] = {{"rope", CALL(rope), nullptr},           {"append", CALL(append), nullptr},
                         {"attention", CALL(attention), nullptr}, {"head_loss", CALL(head_loss), nullptr},
                         {"setup", CALL(setup), nullptr},         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "qlora_decoder_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_qlora_decoder_binding() { return PyModule_Create(&module); }
