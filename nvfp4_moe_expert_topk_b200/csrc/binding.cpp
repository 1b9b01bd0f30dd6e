// binding.cpp -- argument marshalling of the layer operators' Python entry
// points (norm, few-row products, balance loss).  A single-token call of these
// takes about 3 us on the device.  Checking eight tensors and passing their
// pointers from Python takes 5 us on top of the launch, so that the host, not
// the device, would set the pace of a decode step; here it takes under 1 us
// (one row of 7168 elements, called in a loop: 8.3 -> 4.1 us a call).
// No arithmetic: each function checks its tensors (the ValueError says what is
// wrong), takes their pointers and the current stream of their device, and
// calls the C entry point whose address `bind` was given.  Returns the status
// code.  No C++ exception leaves a function.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "nvfp4moe.h"

namespace {

struct Refusal {
    std::string text;
};

struct PythonError {};      // the interpreter's error is set

decltype(&nvfp4_add_rmsnorm) f_norm = nullptr;
decltype(&nvfp4_gemv) f_gemv = nullptr;
decltype(&nvfp4_moe_balance) f_balance = nullptr;
decltype(&nvfp4_moe_balance_backward) f_backward = nullptr;

inline std::string text(const char *s) { return s; }
inline std::string text(const std::string &s) { return s; }
inline std::string text(int64_t v) { return std::to_string(v); }
inline std::string text(int v) { return std::to_string(v); }

template <typename... A>
[[noreturn]] void refuse(const A &...a)
{
    throw Refusal{(std::string() + ... + text(a))};
}

std::string shape_text(c10::IntArrayRef s)
{
    std::string o = "[";
    for (size_t i = 0; i < s.size(); ++i)
        o += (i ? ", " : "") + std::to_string(s[i]);
    return o + "]";
}

const char *type_text(at::ScalarType t)
{
    switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kLong: return "torch.int64";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
    }
}

// The CUDA tensor `o`; on device `dev` where dev >= 0.
const at::Tensor &tensor(PyObject *o, const char *name, int dev)
{
    if (o == Py_None)
        refuse(name, " is required");
    if (!THPVariable_Check(o))
        refuse(name, " must be a CUDA tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != c10::kStrided)
        refuse(name, " must be a CUDA tensor");
    if (dev >= 0 && t.get_device() != dev)
        refuse(name, " must be a CUDA tensor on cuda:", dev, ", got cuda:", static_cast<int>(t.get_device()));
    return t;
}

void of_type(const at::Tensor &t, const char *name, at::ScalarType type)
{
    if (t.scalar_type() != type)
        refuse(name, " must be ", type_text(type), ", got ", type_text(t.scalar_type()));
}

// Pointer of a contiguous tensor of n elements (n < 0: any number).
template <typename T>
T *flat(PyObject *o, const char *name, int dev, at::ScalarType type, int64_t n)
{
    const at::Tensor &t = tensor(o, name, dev);
    of_type(t, name, type);
    if (!t.is_contiguous())
        refuse(name, " must be contiguous");
    if (n >= 0 && t.numel() != n)
        refuse(name, " must hold ", n, " elements, got ", t.numel());
    return static_cast<T *>(t.data_ptr());
}

// Pointer and row stride of a bf16 matrix [r, c] whose rows may be strided.
uint16_t *rows(PyObject *o, const char *name, int dev, int64_t r, int64_t c, int64_t &ld)
{
    const at::Tensor &t = tensor(o, name, dev);
    of_type(t, name, at::kBFloat16);
    if (t.dim() != 2 || t.size(0) != r || t.size(1) != c)
        refuse(name, " must be [", r, ", ", c, "], got ", shape_text(t.sizes()));
    if (t.is_contiguous()) {
        ld = c;
    } else {
        if (t.stride(1) != 1 && c > 1)
            refuse(name, " must have unit stride along its rows");
        ld = t.stride(0);
    }
    return static_cast<uint16_t *>(t.data_ptr());
}

int64_t integer(PyObject *o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw PythonError{};
    return v;
}

int small(PyObject *o, const char *name)
{
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX)
        refuse(name, " is out of range: ", v);
    return static_cast<int>(v);
}

// The launch's stream: the given one (it has to be on `dev`), or dev's current.
void *stream_of(PyObject *o, int dev)
{
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    PyObject *d = PyObject_GetAttrString(o, "device_index"), *s = PyObject_GetAttrString(o, "cuda_stream");
    if (d == nullptr || s == nullptr) {
        Py_XDECREF(d);
        Py_XDECREF(s);
        throw PythonError{};
    }
    const long long di = PyLong_AsLongLong(d);
    void *raw = PyLong_AsVoidPtr(s);
    Py_DECREF(d);
    Py_DECREF(s);
    if (PyErr_Occurred())
        throw PythonError{};
    if (di != dev)
        refuse("the stream is on cuda:", static_cast<int64_t>(di), ", the tensors on cuda:", dev);
    return raw;
}

// Runs `body` and turns what it throws into a Python error.
template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F body)
{
    try {
        if (got != want)
            refuse("expected ", want, " arguments, got ", got);
        return PyLong_FromLong(body());
    } catch (const Refusal &r) {
        PyErr_SetString(PyExc_ValueError, r.text.c_str());
    } catch (const PythonError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// The entry point, called with the interpreter lock released (a launch waits
// where the stream's queue is full).
template <typename F, typename... A>
int call(F *f, A... a)
{
    PyThreadState *state = PyEval_SaveThread();
    const int status = f(a...);
    PyEval_RestoreThread(state);
    return status;
}

// bind(addresses of the four entry points)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 4, [&] {
        f_norm = reinterpret_cast<decltype(f_norm)>(PyLong_AsVoidPtr(a[0]));
        f_gemv = reinterpret_cast<decltype(f_gemv)>(PyLong_AsVoidPtr(a[1]));
        f_balance = reinterpret_cast<decltype(f_balance)>(PyLong_AsVoidPtr(a[2]));
        f_backward = reinterpret_cast<decltype(f_backward)>(PyLong_AsVoidPtr(a[3]));
        if (PyErr_Occurred())
            throw PythonError{};
        return 0;
    });
}

// add_rmsnorm(x, weight, eps, y, residual, residual_out, quant, gs, codes, scales, scale_layout, stream)
PyObject *add_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 12, [&] {
        const at::Tensor &x = tensor(a[0], "x", -1);
        if (x.dim() != 2)
            refuse("x must be [T, H], got ", shape_text(x.sizes()));
        const int dev = x.get_device();
        nvfp4_norm_args p{};
        p.T = x.size(0);
        p.H = x.size(1);
        p.x = rows(a[0], "x", dev, p.T, p.H, p.ldx);
        p.weight = flat<uint16_t>(a[1], "weight", dev, at::kBFloat16, p.H);
        p.eps = PyFloat_AsDouble(a[2]);
        if (PyErr_Occurred())
            throw PythonError{};
        p.quant = small(a[6], "quant");
        p.scale_layout = small(a[10], "scale_layout");
        if ((a[4] == Py_None) != (a[5] == Py_None))
            refuse("residual and residual_out come together");
        if (a[4] != Py_None) {
            p.residual = rows(a[4], "residual", dev, p.T, p.H, p.ldr);
            p.residual_out = rows(a[5], "residual_out", dev, p.T, p.H, p.ldro);
        }
        if (a[3] != Py_None)
            p.y = rows(a[3], "y", dev, p.T, p.H, p.ldy);
        else if (p.quant == NVFP4_QUANT_NONE)
            refuse("y is required without a quantised output");
        if (p.quant == NVFP4_QUANT_NVFP4) {
            p.gs = flat<float>(a[7], "gs", dev, at::kFloat, 1);
            p.codes = flat<uint8_t>(a[8], "codes", dev, at::kByte, p.T * (p.H / 2));
            p.scales = flat<uint8_t>(a[9], "scales", dev, at::kByte, -1);
            const int64_t padded = p.scale_layout == NVFP4_SCALES_ROWMAJOR ? p.T : (p.T + 127) / 128 * 128;
            const int64_t have = THPVariable_Unpack(a[9]).numel();
            if (have < padded * (p.H / 16))
                refuse("scales must hold ", padded * (p.H / 16), " bytes, got ", have);
        } else if (p.quant == NVFP4_QUANT_E4M3) {
            const bool f8 = THPVariable_Check(a[8]) && THPVariable_Unpack(a[8]).scalar_type() == at::kFloat8_e4m3fn;
            p.codes = flat<uint8_t>(a[8], "codes", dev, f8 ? at::kFloat8_e4m3fn : at::kByte, p.T * p.H);
            p.scales = flat<float>(a[9], "scales", dev, at::kFloat, p.T * ((p.H + 127) / 128));
        }
        void *s = stream_of(a[11], dev);
        const c10::cuda::OptionalCUDAGuard guard(x.device());
        return call(f_norm, &p, s);
    });
}

// gemv(x, b_codes, b_scales, b_gs, seg_end, out, stream)
PyObject *gemv(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        const at::Tensor &x = tensor(a[0], "x", -1);
        if (x.dim() != 2)
            refuse("x must be [M, K], got ", shape_text(x.sizes()));
        const int dev = x.get_device();
        const int64_t M = x.size(0), K = x.size(1);
        const at::Tensor &codes = tensor(a[1], "b_codes", dev);
        of_type(codes, "b_codes", at::kByte);
        if (codes.dim() < 1)
            refuse("b_codes must be [N, K/2], got ", shape_text(codes.sizes()));
        const int64_t N = codes.size(0);
        int64_t ldx = 0, ldo = 0;
        const uint16_t *px = rows(a[0], "x", dev, M, K, ldx);
        uint16_t *po = rows(a[5], "out", dev, M, N, ldo);
        const uint8_t *pc = flat<uint8_t>(a[1], "b_codes", dev, at::kByte, N * (K / 2));
        const uint8_t *ps = flat<uint8_t>(a[2], "b_scales", dev, at::kByte, -1);
        const int64_t need = (N + 127) / 128 * 128 * (K / 16), have = THPVariable_Unpack(a[2]).numel();
        if (have < need)
            refuse("b_scales must hold ", need, " bytes, got ", have);
        PyObject *seq = PySequence_Fast(a[4], "seg_end must be a sequence of column ends");
        if (seq == nullptr)
            throw PythonError{};
        const Py_ssize_t nseg = PySequence_Fast_GET_SIZE(seq);
        int64_t seg[4] = {0, 0, 0, 0};
        for (Py_ssize_t i = 0; i < nseg && i < 4; ++i)
            seg[i] = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
        Py_DECREF(seq);
        if (PyErr_Occurred())
            throw PythonError{};
        const float *pg = flat<float>(a[3], "b_gs", dev, at::kFloat, nseg);
        void *s = stream_of(a[6], dev);
        const c10::cuda::OptionalCUDAGuard guard(x.device());
        // (more than four segments: refused by the entry point before it reads their ends)
        return call(f_gemv, px, M, ldx, pc, ps, pg, seg, static_cast<int>(nseg < 5 ? nseg : 5), N, K, po, ldo, s);
    });
}

// What both directions of the balance loss take.
struct Balance {
    int dev, E, k, scoring;
    int64_t T, ld, S = 1;
    const float *logits;
    const int32_t *ids, *offsets = nullptr;

    Balance(PyObject *l, PyObject *i, PyObject *kk, PyObject *off, PyObject *sc)
    {
        const at::Tensor &t = tensor(l, "logits", -1);
        dev = t.get_device();
        logits = flat<float>(l, "logits", dev, at::kFloat, -1);
        if (t.dim() != 2)
            refuse("logits must be [T, E], got ", shape_text(t.sizes()));
        T = t.size(0);
        if (t.size(1) > INT32_MAX)
            refuse("logits must be [T, E], got ", shape_text(t.sizes()));
        E = static_cast<int>(t.size(1));
        k = small(kk, "k");
        scoring = small(sc, "scoring");
        ids = flat<int32_t>(i, "topk_ids", dev, at::kInt, -1);
        const at::Tensor &d = THPVariable_Unpack(i);
        if (d.dim() != 2 || d.size(0) != T || d.size(1) < k)
            refuse("topk_ids must be [", T, ", >= ", k, "], got ", shape_text(d.sizes()));
        ld = d.size(1);
        if (off != Py_None) {
            offsets = flat<int32_t>(off, "seq_offsets", dev, at::kInt, -1);
            S = THPVariable_Unpack(off).numel() - 1;
            if (S < 1)
                refuse("seq_offsets must hold at least 2 elements, got ", S + 1);
        }
    }
};

// balance(logits, ids, k, counts, tokens, probs, loss, workspace, seq_offsets, scoring, stream)
PyObject *balance(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const Balance b(a[0], a[1], a[2], a[8], a[9]);
        int32_t *counts = flat<int32_t>(a[3], "counts", b.dev, at::kInt, b.S * b.E);
        int32_t *tokens = flat<int32_t>(a[4], "tokens", b.dev, at::kInt, b.S);
        float *probs = flat<float>(a[5], "probs", b.dev, at::kFloat, b.S * b.E);
        float *loss = flat<float>(a[6], "loss", b.dev, at::kFloat, b.S);
        uint8_t *ws = flat<uint8_t>(a[7], "workspace", b.dev, at::kByte, -1);
        const int64_t bytes = THPVariable_Unpack(a[7]).numel();
        void *s = stream_of(a[10], b.dev);
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(b.dev)));
        return call(f_balance, b.logits, b.ids, b.ld, b.T, b.E, b.k, b.offsets, b.S, b.scoring, counts, tokens, probs, loss,
                         ws, static_cast<size_t>(bytes), s);
    });
}

// backward(logits, ids, k, counts, tokens, grad_loss, grad_logits, grad_weights, seq_offsets, scoring, stream)
PyObject *backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const Balance b(a[0], a[1], a[2], a[8], a[9]);
        const int32_t *counts = flat<int32_t>(a[3], "counts", b.dev, at::kInt, b.S * b.E);
        const int32_t *tokens = flat<int32_t>(a[4], "tokens", b.dev, at::kInt, b.S);
        const float *gl = flat<float>(a[5], "grad_loss", b.dev, at::kFloat, b.S);
        float *out = flat<float>(a[6], "grad_logits", b.dev, at::kFloat, b.T * b.E);
        const float *gw = a[7] == Py_None ? nullptr : flat<float>(a[7], "grad_weights", b.dev, at::kFloat, b.T * b.k);
        void *s = stream_of(a[10], b.dev);
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(b.dev)));
        return call(f_backward, b.logits, b.ids, b.ld, b.T, b.E, b.k, b.offsets, b.S, b.scoring, counts, tokens, gl, gw, out, s);
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast()
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(F));
}

PyMethodDef methods[] = {
    {"bind", fast<bind>(), METH_FASTCALL, "Addresses of the C entry points."},
    {"add_rmsnorm", fast<add_rmsnorm>(), METH_FASTCALL, "nvfp4_add_rmsnorm's status."},
    {"gemv", fast<gemv>(), METH_FASTCALL, "nvfp4_gemv's status."},
    {"balance", fast<balance>(), METH_FASTCALL, "nvfp4_moe_balance's status."},
    {"backward", fast<backward>(), METH_FASTCALL, "nvfp4_moe_balance_backward's status."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Argument marshalling of the layer operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__binding(void)
{
    return PyModule_Create(&module);
}
