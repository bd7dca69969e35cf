// Native marshalling of the calls that a decode step or a short prompt makes eagerly, one
// after another: lora_quant_i8, lora_linear_i8, lora_linear_i8_sgmv, lora_rope.  Their
// kernels take 2 to 20 us; reading the arguments' attributes from Python and converting them
// with ctypes took 6 to 9 us a call (22 with a pool: 9 here), one launch 2.5.  This file checks
// the same things on the tensors' C++ side and calls the same C ABI (its entry points are
// handed in, so the library is loaded in one place only).

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <map>
#include <utility>

#include "lora_sgmv.h"

namespace {

PyObject *g_error = nullptr;            // LoraError(what, code)
PyObject *g_new_workspace = nullptr;    // (device, stream or None, bytes) -> Workspace
decltype(&lora_quant_i8) g_quant = nullptr;
decltype(&lora_linear_i8) g_linear = nullptr;
decltype(&lora_rope) g_rope = nullptr;
decltype(&lora_linear_i8_sgmv) g_sgmv = nullptr;
decltype(&lora_workspace_size) g_workspace_size = nullptr;

struct Refused {                        // thrown inside a call, raised as LoraError at its end
    const char *what;
    int code;
};

struct Workspace {                      // the workspace of a device and stream, kept until a larger one is needed
    PyObject *object = nullptr;
    void *at = nullptr;
    size_t bytes = 0;
    unsigned long long stream_id = 0;   // (a stream destroyed and a new one may have the same handle)
};
std::map<std::pair<int, cudaStream_t>, Workspace> g_workspaces;

const at::Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o))
        throw Refused{what, LORA_ERR_INVALID_ARG};
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != c10::kStrided)
        throw Refused{"tensors must be dense and live on one CUDA device", LORA_ERR_INVALID_ARG};
    return t;
}

int device_of(const at::Tensor &t, int dev)
{
    const int d = t.get_device();
    if (dev >= 0 && d != dev)
        throw Refused{"tensors must live on one CUDA device", LORA_ERR_INVALID_ARG};
    return d;
}

// Leading dimension of a matrix [n, d] (a single row has none: any that fits will do).
int64_t rows(const at::Tensor &t, int64_t n, int64_t d, const char *what)
{
    if (t.dim() != 2 || t.size(0) != n || t.size(1) != d || (d > 1 && t.stride(1) != 1))
        throw Refused{what, LORA_ERR_INVALID_ARG};
    return n > 1 ? t.stride(0) : (d + 15) / 16 * 16;
}

const float *scales(const at::Tensor &t, int64_t n, const char *what)
{
    if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
        throw Refused{what, LORA_ERR_INVALID_ARG};
    return static_cast<const float *>(t.data_ptr());
}

int32_t dtype(const at::Tensor &t)
{
    switch (t.scalar_type()) {
    case at::kBFloat16:
        return LORA_BF16;
    case at::kHalf:
        return LORA_F16;
    case at::kFloat:
        return LORA_F32;
    default:
        throw Refused{"bf16, fp16 or fp32 expected", LORA_ERR_UNSUPPORTED};
    }
}

int32_t as_i32(int64_t v)
{
    if (v != (int32_t)v)
        throw Refused{"sizes must fit 32 bits", LORA_ERR_UNSUPPORTED};
    return (int32_t)v;
}

// The stream object's handle, or the device's current stream.
cudaStream_t stream_of(PyObject *o, int dev)
{
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream(dev).stream();
    PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h)
        throw std::exception();          // (the Python error stands)
    void *p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred())
        throw std::exception();
    return static_cast<cudaStream_t>(p);
}

Workspace read_workspace(PyObject *o)
{
    PyObject *at = PyObject_CallMethod(o, "ptr", nullptr), *n = at ? PyObject_GetAttrString(o, "nbytes") : nullptr;
    Workspace w;
    w.object = o;
    if (at && n) {
        w.at = PyLong_AsVoidPtr(at);
        w.bytes = PyLong_AsSize_t(n);
    }
    Py_XDECREF(at);
    Py_XDECREF(n);
    if (PyErr_Occurred())
        throw std::exception();
    return w;
}

// A workspace that the caller made: its memory has to be the operands' device's (another
// GPU's or the host's would be a bad address inside the kernels).
void check_place(PyObject *given, const Workspace &w, int dev)
{
    PyObject *t = PyObject_GetAttrString(given, "tensor");
    int at = -1;
    if (t && THPVariable_Check(t)) {
        const at::Tensor &v = THPVariable_Unpack(t);
        at = v.is_cuda() ? v.get_device() : -1;
    } else {                             // (some other object with ptr() and nbytes)
        cudaPointerAttributes a = {};
        if (cudaPointerGetAttributes(&a, w.at) != cudaSuccess)
            cudaGetLastError();
        else if (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged)
            at = a.device;
    }
    PyErr_Clear();
    Py_XDECREF(t);
    if (at != dev)
        throw Refused{"the workspace must live on the tensors' device", LORA_ERR_INVALID_ARG};
}

// Waits for all of the device's work, whatever its streams.
void device_idle()
{
    // (a capture of another thread does not forbid it)
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    cudaError_t e = cudaSuccess;
    Py_BEGIN_ALLOW_THREADS
    e = cudaDeviceSynchronize();
    Py_END_ALLOW_THREADS
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) {
        cudaGetLastError();
        throw Refused{"cudaDeviceSynchronize", LORA_ERR_CUDA};
    }
}

// A new reference to the call's workspace: the one given, else this device and stream's;
// under graph capture a fresh one from the graph's memory, so that no two graphs share it.
Workspace workspace(PyObject *given, PyObject *stream, int dev, cudaStream_t s, size_t bytes)
{
    if (given != Py_None) {
        Workspace w = read_workspace(given);
        check_place(given, w, dev);
        Py_INCREF(given);
        return w;
    }
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &capturing) != cudaSuccess) {
        cudaGetLastError();
        capturing = cudaStreamCaptureStatusNone;
    }
    const std::pair<int, cudaStream_t> key(dev, s);
    unsigned long long id = 0;
    if (capturing == cudaStreamCaptureStatusNone) {
        if (cudaStreamGetId(s, &id) != cudaSuccess)
            cudaGetLastError();
        auto it = g_workspaces.find(key);
        if (it != g_workspaces.end() && it->second.stream_id != id) {
            device_idle();                   // the stream that used it is gone, its work may not be
            it = g_workspaces.find(key);
            if (it != g_workspaces.end())
                it->second.stream_id = id;
        }
        if (it != g_workspaces.end()) {
            if (it->second.bytes >= bytes) {
                Py_INCREF(it->second.object);
                return it->second;
            }
            bytes = std::max(bytes, 2 * it->second.bytes);
        }
    }
    PyObject *o = PyObject_CallFunction(g_new_workspace, "iOn", dev, stream, (Py_ssize_t)bytes);
    if (!o)
        throw std::exception();
    Workspace w;
    try {
        w = read_workspace(o);
    } catch (...) {
        Py_DECREF(o);
        throw;
    }
    if (capturing == cudaStreamCaptureStatusNone) {
        Py_INCREF(o);
        Workspace &kept = g_workspaces[key];
        PyObject *old = kept.object;
        kept = w;
        kept.stream_id = id;
        Py_XDECREF(old);
    }
    return w;
}

PyObject *raise(const char *what, int code)
{
    PyObject *e = PyObject_CallFunction(g_error, "si", what, code);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

// Runs f; whatever it throws leaves as a Python exception.
template <class F> PyObject *guarded(F f)
{
    try {
        return f();
    } catch (const Refused &r) {
        return raise(r.what, r.code);
    } catch (const std::exception &e) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

bool takes(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want)
        return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return false;
}

// quant_i8(X, Q, S, stream)
PyObject *quant_i8(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    if (!takes(n_args, 4))
        return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &X = tensor(a[0], "X must be a tensor"), &Q = tensor(a[1], "Q must be a tensor"),
                         &S = tensor(a[2], "S must be a tensor");
        const int dev = device_of(S, device_of(Q, device_of(X, -1)));
        if (X.dim() != 2 || Q.scalar_type() != at::kChar)
            throw Refused{"X must be a matrix, Q an int8 one", LORA_ERR_INVALID_ARG};
        const int64_t n = X.size(0), d = X.size(1);
        const int64_t ldx = rows(X, n, d, "X must have unit-stride columns");
        const int64_t ldq = rows(Q, n, d, "Q must have X's shape and unit-stride columns");
        const float *s = scales(S, n, "S must be a contiguous fp32 tensor, one scale a row");
        const int32_t t = dtype(X), n32 = as_i32(n), d32 = as_i32(d);
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != dev)
            guard.set_index(dev);
        const int rc = g_quant(X.data_ptr(), t, ldx, static_cast<int8_t *>(Q.data_ptr()), ldq, const_cast<float *>(s),
                               n32, d32, stream_of(a[3], dev));
        if (rc != LORA_OK)
            return raise("lora_quant_i8", rc);
        Py_RETURN_NONE;
    });
}

// The operands of a projection with an 8-bit weight.
struct I8 {
    int dev;
    int64_t ldq, ldw, ldy;
    const int8_t *q, *w;
    const float *sx, *sw;
    void *y;
    int32_t type, n, d_in, d_out;

    I8(PyObject *oq, PyObject *osx, PyObject *ow, PyObject *osw, PyObject *oy)
    {
        const at::Tensor &Q = tensor(oq, "Q must be a tensor"), &Sx = tensor(osx, "Sx must be a tensor"),
                         &W = tensor(ow, "Wq must be a tensor"), &Sw = tensor(osw, "Sw must be a tensor"),
                         &Y = tensor(oy, "Y must be a tensor");
        dev = device_of(Y, device_of(Sw, device_of(W, device_of(Sx, device_of(Q, -1)))));
        if (Q.scalar_type() != at::kChar || W.scalar_type() != at::kChar || Q.dim() != 2 || W.dim() != 2 ||
            Q.size(1) != W.size(1))
            throw Refused{"Q [N, d_in] and Wq [d_out, d_in] must be int8 matrices", LORA_ERR_INVALID_ARG};
        n = as_i32(Q.size(0));
        d_in = as_i32(Q.size(1));
        d_out = as_i32(W.size(0));
        ldq = rows(Q, n, d_in, "Q must have unit-stride columns");
        ldw = rows(W, d_out, d_in, "Wq must have unit-stride columns");
        ldy = rows(Y, n, d_out, "Y must be [N, d_out] with unit-stride columns");
        sx = scales(Sx, n, "Sx must be a contiguous fp32 tensor, one scale a token");
        sw = scales(Sw, d_out, "Sw must be a contiguous fp32 tensor, one scale a channel");
        q = static_cast<const int8_t *>(Q.data_ptr());
        w = static_cast<const int8_t *>(W.data_ptr());
        y = Y.data_ptr();
        type = dtype(Y);
    }
};

// linear_i8(Q, Sx, Wq, Sw, Y, workspace or None, stream) -> workspace
PyObject *linear_i8(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    if (!takes(n_args, 7))
        return nullptr;
    return guarded([&]() -> PyObject * {
        const I8 o(a[0], a[1], a[2], a[3], a[4]);
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != o.dev)
            guard.set_index(o.dev);
        const cudaStream_t s = stream_of(a[6], o.dev);
        const Workspace ws = workspace(a[5], a[6], o.dev, s, 256);
        const int rc = g_linear(o.q, o.ldq, o.sx, o.w, o.ldw, o.sw, o.y, o.type, o.ldy, o.n, o.d_in, o.d_out, ws.at,
                                ws.bytes, s);
        if (rc != LORA_OK) {
            Py_DECREF(ws.object);
            return raise("lora_linear_i8", rc);
        }
        return ws.object;
    });
}

// A pool object's tensors and sizes (the attributes hold the references).
struct Pool {
    PyObject *held[5] = {};
    lora_pool p = {};

    Pool(PyObject *o, PyObject *max_rank, int dev)
    {
        static const char *const names[5] = {"A", "B", "A_off", "B_off", "rank"};
        static const char *const wrong[5] = {"pool.A must be contiguous bf16", "pool.B must be contiguous bf16",
                                             "pool.A_off must be contiguous int64", "pool.B_off must be contiguous int64",
                                             "pool.rank must be contiguous int32"};
        const at::ScalarType types[5] = {at::kBFloat16, at::kBFloat16, at::kLong, at::kLong, at::kInt};
        const void *ptr[5];
        int64_t n[5];
        try {
            for (int i = 0; i < 5; ++i) {
                if (!(held[i] = PyObject_GetAttrString(o, names[i])))
                    throw std::exception();
                const at::Tensor &t = tensor(held[i], wrong[i]);
                device_of(t, dev);
                if (t.scalar_type() != types[i] || !t.is_contiguous())
                    throw Refused{wrong[i], LORA_ERR_INVALID_ARG};
                ptr[i] = t.data_ptr();
                n[i] = t.numel();
            }
            p.A = ptr[0];
            p.B = ptr[1];
            p.A_off = static_cast<const int64_t *>(ptr[2]);
            p.B_off = static_cast<const int64_t *>(ptr[3]);
            p.rank = static_cast<const int32_t *>(ptr[4]);
            p.A_elems = n[0];
            p.B_elems = n[1];
            if (n[2] < n[4] || n[3] < n[4])
                throw Refused{"pool.A_off and pool.B_off need an entry for every rank", LORA_ERR_INVALID_ARG};
            p.n_adapters = as_i32(n[4]);
            p.d_in = size(o, "d_in");
            p.d_out = size(o, "d_out");
            p.max_rank = max_rank == Py_None ? size(o, "max_rank") : as_i32(PyLong_AsLongLong(max_rank));
            if (PyErr_Occurred())
                throw std::exception();
        } catch (...) {
            drop();
            throw;
        }
    }
    ~Pool() { drop(); }
    Pool(const Pool &) = delete;

private:
    static int32_t size(PyObject *o, const char *name)
    {
        PyObject *v = PyObject_GetAttrString(o, name);
        if (!v)
            throw std::exception();
        const long long x = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (PyErr_Occurred())
            throw std::exception();
        return as_i32(x);
    }
    void drop()
    {
        for (PyObject *&h : held)
            Py_CLEAR(h);
    }
};

const int32_t *ints(const at::Tensor &t, int64_t least, const char *what)
{
    if (t.scalar_type() != at::kInt || t.numel() < least || !t.is_contiguous())
        throw Refused{what, LORA_ERR_INVALID_ARG};
    return static_cast<const int32_t *>(t.data_ptr());
}

// linear_i8_sgmv(Q, Sx, X, Wq, Sw, Y, pool, seg_off, seg_ad, scale, workspace or None, stream, max_rank or None)
PyObject *linear_i8_sgmv(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    if (!takes(n_args, 13))
        return nullptr;
    return guarded([&]() -> PyObject * {
        const I8 o(a[0], a[1], a[3], a[4], a[5]);
        const at::Tensor &X = tensor(a[2], "X must be a tensor"), &off = tensor(a[7], "seg_off must be a tensor"),
                         &ad = tensor(a[8], "seg_ad must be a tensor");
        device_of(ad, device_of(off, device_of(X, o.dev)));
        if (X.scalar_type() != at::kBFloat16 || o.type != LORA_BF16)
            throw Refused{"X and Y must be bf16", LORA_ERR_INVALID_ARG};
        const int64_t ldx = rows(X, o.n, o.d_in, "X must be [N, d_in] with unit-stride columns");
        const Pool pool(a[6], a[12], o.dev);
        if (pool.p.d_in != o.d_in || pool.p.d_out != o.d_out)
            throw Refused{"Wq must be [pool.d_out, pool.d_in]", LORA_ERR_INVALID_ARG};
        const int32_t n_seg = as_i32(ad.numel());
        const int32_t *seg_ad = ints(ad, n_seg, "seg_ad must be a contiguous int32 tensor");
        const int32_t *seg_off = ints(off, (int64_t)n_seg + 1, "seg_off must be a contiguous int32 tensor of n_seg + 1");
        const double scale = PyFloat_AsDouble(a[9]);
        if (PyErr_Occurred())
            throw std::exception();
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != o.dev)
            guard.set_index(o.dev);
        const cudaStream_t s = stream_of(a[11], o.dev);
        // (sizes the call refuses need none)
        const size_t need = g_workspace_size(LORA_OP_LINEAR_I8_SGMV, o.n, pool.p.n_adapters, o.d_in, o.d_out,
                                             pool.p.max_rank, n_seg, 1);
        const Workspace ws = workspace(a[10], a[11], o.dev, s, std::max<size_t>(need, 256));
        const int rc = g_sgmv(o.q, o.ldq, o.sx, X.data_ptr(), ldx, o.w, o.ldw, o.sw, o.y, o.ldy, &pool.p, seg_off, seg_ad,
                              n_seg, o.n, (float)scale, ws.at, ws.bytes, s);
        if (rc != LORA_OK) {
            Py_DECREF(ws.object);
            return raise("lora_linear_i8_sgmv", rc);
        }
        return ws.object;
    });
}

// rope(xs, ys, pos, freqs, interleaved, mscale, inverse, stream); xs and ys are sequences
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    if (!takes(n_args, 8))
        return nullptr;
    PyObject *xs = PySequence_Fast(a[0], "xs must be a sequence of tensors");
    PyObject *ys = xs ? PySequence_Fast(a[1], "ys must be a sequence of tensors") : nullptr;
    PyObject *done = !ys ? nullptr : guarded([&]() -> PyObject * {
        const Py_ssize_t k = PySequence_Fast_GET_SIZE(xs);
        if (k < 1 || k != PySequence_Fast_GET_SIZE(ys))
            throw Refused{"one output per input", LORA_ERR_INVALID_ARG};
        if (k > LORA_MAX_PROJ)
            throw Refused{"too many tensors", LORA_ERR_UNSUPPORTED};
        const at::Tensor &pos = tensor(a[2], "pos must be a tensor"), &freqs = tensor(a[3], "freqs must be a tensor");
        int dev = device_of(freqs, device_of(pos, -1));
        lora_rope_mat mats[LORA_MAX_PROJ];
        int64_t n = 0, dim = 0;
        int32_t t = 0;
        for (Py_ssize_t i = 0; i < k; ++i) {
            const at::Tensor &x = tensor(PySequence_Fast_GET_ITEM(xs, i), "xs must be tensors"),
                             &y = tensor(PySequence_Fast_GET_ITEM(ys, i), "ys must be tensors");
            dev = device_of(y, device_of(x, dev));
            if (x.dim() != 3)
                throw Refused{"tensors must be [N, heads, dim]", LORA_ERR_INVALID_ARG};
            if (i == 0) {
                n = x.size(0);
                dim = x.size(2);
                t = dtype(x);
            }
            if (x.size(0) != n || x.size(2) != dim || x.sizes() != y.sizes() || dtype(x) != t ||
                x.scalar_type() != y.scalar_type())
                throw Refused{"tensors [N, heads, dim] of one type, N and dim", LORA_ERR_INVALID_ARG};
            if (x.stride(2) != 1 || y.stride(2) != 1)
                throw Refused{"unit stride inside a head", LORA_ERR_INVALID_ARG};
            mats[i] = {x.data_ptr(), y.data_ptr(), x.stride(0), x.stride(1), y.stride(0), y.stride(1), as_i32(x.size(1))};
        }
        const bool wide = pos.scalar_type() == at::kLong;
        if ((!wide && pos.scalar_type() != at::kInt) || pos.dim() != 1 || pos.size(0) != n || (n > 1 && pos.stride(0) != 1))
            throw Refused{"pos must be a contiguous int32 or int64 tensor [N]", LORA_ERR_INVALID_ARG};
        if (freqs.scalar_type() != at::kDouble || freqs.dim() != 1 || !freqs.is_contiguous())
            throw Refused{"freqs must be a contiguous fp64 tensor [rot / 2]", LORA_ERR_INVALID_ARG};
        const int interleaved = PyObject_IsTrue(a[4]), inverse = PyObject_IsTrue(a[6]);
        const double m = PyFloat_AsDouble(a[5]);
        if (PyErr_Occurred())
            throw std::exception();
        const int32_t n32 = as_i32(n), d32 = as_i32(dim), rot = as_i32(2 * freqs.size(0));
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != dev)
            guard.set_index(dev);
        const int rc = g_rope(mats, (int32_t)k, t, pos.data_ptr(), wide ? 8 : 4,
                              static_cast<const double *>(freqs.data_ptr()), n32, d32, rot, interleaved, inverse,
                              (float)m, stream_of(a[7], dev));
        if (rc != LORA_OK)
            return raise("lora_rope", rc);
        Py_RETURN_NONE;
    });
    Py_XDECREF(xs);
    Py_XDECREF(ys);
    return done;
}

// setup(LoraError, new_workspace, addresses of lora_quant_i8, lora_linear_i8, lora_rope,
// lora_linear_i8_sgmv and lora_workspace_size)
PyObject *setup(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    if (!takes(n_args, 7))
        return nullptr;
    void *f[5];
    for (int i = 0; i < 5; ++i)
        f[i] = PyLong_AsVoidPtr(a[2 + i]);
    if (PyErr_Occurred())
        return nullptr;
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    g_error = a[0];
    g_new_workspace = a[1];
    g_quant = reinterpret_cast<decltype(g_quant)>(f[0]);
    g_linear = reinterpret_cast<decltype(g_linear)>(f[1]);
    g_rope = reinterpret_cast<decltype(g_rope)>(f[2]);
    g_sgmv = reinterpret_cast<decltype(g_sgmv)>(f[3]);
    g_workspace_size = reinterpret_cast<decltype(g_workspace_size)>(f[4]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {{"setup", FAST(setup), nullptr},
                           {"quant_i8", FAST(quant_i8), nullptr},
                           {"linear_i8", FAST(linear_i8), nullptr},
                           {"linear_i8_sgmv", FAST(linear_i8_sgmv), nullptr},
                           {"rope", FAST(rope), nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&g_module); }
