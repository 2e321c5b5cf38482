// mq_torch.cpp -- the binding of the calls whose kernels run for a few
// microseconds (mq_linear_w4a16, mq_rope_kv_append, mq_kv_attention): the
// checks and the marshalling of mq.py's other calls, natively, because in
// Python they take longer than the kernels (10.6 us of host time for an append
// through ctypes); and what mq.py asks about streams for its workspaces.  It calls
// the library that mq.py has loaded (release or debug build) through the
// addresses given to bind(), and holds nothing else.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAException.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mq.h"

namespace {

using LinearFn = decltype(&mq_linear_w4a16);
using AppendFn = decltype(&mq_rope_kv_append);
using AttentionFn = decltype(&mq_kv_attention);
LinearFn g_linear = nullptr;
AppendFn g_append = nullptr;
AttentionFn g_attention = nullptr;

// Raised as a Python ValueError.
struct Refused {
    std::string why;
};

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw Refused{std::string(what) + ": tensor expected"};
    return THPVariable_Unpack(o);
}

// The current device, which has to be the tensor's (the library enqueues there).
int device_of(const at::Tensor& t, const char* what) {
    if (!t.is_cuda()) throw Refused{std::string(what) + ": device tensor expected"};
    const int dev = c10::cuda::current_device();
    if (t.get_device() != dev)
        throw Refused{std::string(what) + ": on cuda:" + std::to_string(t.get_device()) +
                      ", but the current device is cuda:" + std::to_string(dev)};
    return dev;
}

const at::Tensor& need(PyObject* o, const char* what, at::ScalarType type, int dev) {
    const at::Tensor& t = tensor(o, what);
    if (t.scalar_type() != type)
        throw Refused{std::string(what) + ": " + c10::toString(type) + " expected, got " + c10::toString(t.scalar_type())};
    if (!t.is_cuda() || t.get_device() != dev)
        throw Refused{std::string(what) + ": expected on cuda:" + std::to_string(dev)};
    if (!t.is_contiguous()) throw Refused{std::string(what) + ": contiguous tensor expected"};
    return t;
}

template <typename T = void>
T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

// Elements between rows of a bf16 tensor [rows, ...] whose rows hold `width`
// consecutive elements (rows may be apart).
int64_t row_stride(const at::Tensor& t, const char* what, int64_t width) {
    if (t.scalar_type() != at::kBFloat16) throw Refused{std::string(what) + ": BFloat16 expected"};
    int64_t expect = 1;
    for (int64_t d = t.dim() - 1; d > 0; --d) {
        if (t.size(d) != 1 && t.stride(d) != expect)
            throw Refused{std::string(what) + ": consecutive elements within a row expected"};
        expect *= t.size(d);
    }
    return t.size(0) > 1 ? t.stride(0) : width;
}

void* stream_of(PyObject* o, int dev) {
    if (o == nullptr || o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
    if (v == nullptr) {
        PyErr_Clear();
        v = Py_NewRef(o);
    }
    void* s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (s == nullptr && PyErr_Occurred()) throw Refused{"stream: a stream or its address expected"};
    return s;
}

struct Kv {
    mq_kv_cache cache;
    mq_kv_batch batch;
};

// args: cu_rows, lens, page_table, k_codes, v_codes, k_scales, v_scales
Kv kv_of(PyObject* const* args, int dev) {
    const at::Tensor& k = tensor(args[3], "k_codes");
    const at::ScalarType codes = k.scalar_type();
    if (codes != at::kFloat8_e4m3fn && codes != at::kByte)
        throw Refused{std::string("k_codes: Float8_e4m3fn or Byte expected, got ") + c10::toString(codes)};
    need(args[3], "k_codes", codes, dev);
    const at::Tensor& v = need(args[4], "v_codes", codes, dev);
    const at::Tensor& ks = need(args[5], "k_scales", at::kFloat, dev);
    const at::Tensor& vs = need(args[6], "v_scales", at::kFloat, dev);
    const at::Tensor& cu = need(args[0], "cu_rows", at::kInt, dev);
    const at::Tensor& lens = need(args[1], "lens", at::kInt, dev);
    const at::Tensor& table = need(args[2], "page_table", at::kInt, dev);
    if (k.dim() != 4 || v.sizes() != k.sizes())
        throw Refused{"k_codes, v_codes: [pages, kv heads, page size, head_dim] expected of both"};
    if (ks.dim() != 2 || ks.size(0) != k.size(0) || ks.size(1) != k.size(1) || vs.sizes() != ks.sizes())
        throw Refused{"k_scales, v_scales: [pages, kv heads] expected"};
    if (table.dim() != 2 || cu.numel() != table.size(0) + 1 || lens.numel() != table.size(0))
        throw Refused{"cu_rows [batch + 1], lens [batch] and page_table [batch, max_pages] do not agree"};
    const int64_t most = 0x7fffffff;
    if (k.size(1) > most || k.size(2) > most || k.size(3) > most || table.size(0) > most)
        throw Refused{"k_codes, page_table: too large"};
    return Kv{{ptr<uint8_t>(k), ptr<uint8_t>(v), ptr<float>(ks), ptr<float>(vs), k.size(0), (int32_t)k.size(2),
               (int32_t)k.size(1), (int32_t)k.size(3), 0},
              {ptr<int32_t>(cu), ptr<int32_t>(lens), ptr<int32_t>(table), table.size(1), (int32_t)table.size(0), 0}};
}

int32_t int32_of(int64_t v, const char* what) {
    if (v < INT32_MIN || v > INT32_MAX) throw Refused{std::string(what) + ": out of range"};
    return (int32_t)v;
}

// Lets other Python threads run while it lives: a launch waits where its
// stream's queue is full.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// Runs f, with its refusals and torch's exceptions as Python errors; false with one.
template <typename F>
bool guarded_void(F f) {
    try {
        f();
        return true;
    } catch (const Refused& r) {
        PyErr_SetString(PyExc_ValueError, r.why.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return false;
}
// The same; f's status as an int.
template <typename F>
PyObject* guarded(F f) {
    int status = 0;
    return guarded_void([&] { status = f(); }) ? PyLong_FromLong(status) : nullptr;
}

PyObject* py_bind(PyObject*, PyObject* args) {
    unsigned long long a, b, c;
    if (!PyArg_ParseTuple(args, "KKK", &a, &b, &c)) return nullptr;
    g_linear = reinterpret_cast<LinearFn>(a);
    g_append = reinterpret_cast<AppendFn>(b);
    g_attention = reinterpret_cast<AttentionFn>(c);
    Py_RETURN_NONE;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    return false;
}

bool number(PyObject* o, long long* v) {
    *v = PyLong_AsLongLong(o);
    return !(*v == -1 && PyErr_Occurred());
}

// x, w_codes, w_scales, alpha_w, N, y, stream
PyObject* py_linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
    long long N;
    if (!count(n, 7) || !number(args[4], &N)) return nullptr;
    return guarded([&] {
        const int dev = device_of(tensor(args[0], "x"), "x");
        const at::Tensor& x = need(args[0], "x", at::kBFloat16, dev);
        const at::Tensor& c = need(args[1], "w_codes", at::kByte, dev);
        const at::Tensor& s = need(args[2], "w_scales", at::kByte, dev);
        const at::Tensor& alpha = need(args[3], "alpha_w", at::kFloat, dev);
        const at::Tensor& y = need(args[5], "y", at::kBFloat16, dev);
        if (x.dim() != 2) throw Refused{"x: [M, K] expected"};
        const int64_t M = x.size(0), K = x.size(1);
        if (N < 0 || c.numel() < N * (K / 2) || s.numel() < (N + 127) / 128 * 128 * ((K + 63) / 64 * 4) || alpha.numel() < 1)
            throw Refused{"w_codes, w_scales, alpha_w: smaller than an [N, K] weight's"};
        if (y.numel() < M * N) throw Refused{"y: smaller than [M, N]"};
        void* stream = stream_of(args[6], dev);
        Unlocked unlocked;
        return g_linear(ptr(x), M, K, ptr<uint8_t>(c), ptr<uint8_t>(s), ptr<float>(alpha), N, ptr(y), stream);
    });
}

// qkv, rope, cu_rows, lens, page_table, k_codes, v_codes, k_scales, v_scales, q_out, ws, rot_dim, interleaved, stream
PyObject* py_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (!count(n, 14)) return nullptr;
    long long rot_dim = -1;
    if (args[11] != Py_None && !number(args[11], &rot_dim)) return nullptr;
    const int interleaved = PyObject_IsTrue(args[12]);
    if (interleaved < 0) return nullptr;
    return guarded([&] {
        const at::Tensor& qkv = tensor(args[0], "qkv");
        const int dev = device_of(qkv, "qkv");
        const Kv kv = kv_of(args + 2, dev);
        const at::Tensor& q = need(args[9], "q_out", at::kBFloat16, dev);
        if (q.dim() != 3 || q.size(2) != kv.cache.head_dim || qkv.dim() != 2 || qkv.size(0) != q.size(0) ||
            qkv.size(1) != (q.size(1) + 2 * kv.cache.kv_heads) * q.size(2))
            throw Refused{"qkv [T, (q heads + 2 kv heads) head_dim] and q_out [T, q heads, head_dim] do not agree"};
        const float* rope = nullptr;
        int64_t positions = 0, columns = 0;
        if (args[1] != Py_None) {
            const at::Tensor& r = need(args[1], "rope", at::kFloat, dev);
            if (r.dim() != 2 || (rot_dim >= 0 && r.size(1) != rot_dim)) throw Refused{"rope: [positions, rot_dim] expected"};
            rope = ptr<float>(r);
            positions = r.size(0);
            columns = r.size(1);
        }
        void* ws = nullptr;
        size_t ws_bytes = 0;
        if (args[10] != Py_None) {
            const at::Tensor& w = need(args[10], "ws", at::kByte, dev);
            ws = ptr(w);
            ws_bytes = (size_t)w.numel();
        }
        const int64_t T = q.size(0), stride = row_stride(qkv, "qkv", qkv.size(1));
        const int32_t heads = int32_of(q.size(1), "q_out"), rot = int32_of(rot_dim >= 0 ? rot_dim : columns, "rot_dim");
        void* stream = stream_of(args[13], dev);
        Unlocked unlocked;
        return g_append(ptr(qkv), T, stride, heads, rope, positions, rot, interleaved, &kv.cache, &kv.batch, ptr(q), ws,
                        ws_bytes, stream);
    });
}

// q, cu_rows, lens, page_table, k_codes, v_codes, k_scales, v_scales, out, ws, max_q, max_len, scale, stream
PyObject* py_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
    long long max_q, max_len;
    if (!count(n, 14) || !number(args[10], &max_q) || !number(args[11], &max_len)) return nullptr;
    const double scale = PyFloat_AsDouble(args[12]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    return guarded([&] {
        const at::Tensor& q = tensor(args[0], "q");
        const int dev = device_of(q, "q");
        const Kv kv = kv_of(args + 1, dev);
        const at::Tensor& out = need(args[8], "out", at::kBFloat16, dev);
        const at::Tensor& ws = need(args[9], "ws", at::kByte, dev);
        if (q.dim() != 3 || q.size(2) != kv.cache.head_dim || out.sizes() != q.sizes())
            throw Refused{"q and out [T, q heads, head_dim] do not agree with the cache"};
        const int64_t T = q.size(0), stride = row_stride(q, "q", q.size(1) * q.size(2));
        const int32_t heads = int32_of(q.size(1), "q");
        void* stream = stream_of(args[13], dev);
        Unlocked unlocked;
        return g_attention(ptr(q), T, stride, heads, &kv.cache, &kv.batch, max_q, max_len, (float)scale, ptr(out), ptr(ws),
                           (size_t)ws.numel(), stream);
    });
}

// stream, device -> what a workspace belongs to: (device index, the stream's
// address, the id of the graph capture that the stream is in, 0 for none)
PyObject* py_place(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (!count(n, 2)) return nullptr;
    int index = 0;
    void* stream = nullptr;
    unsigned long long id = 0;
    if (!guarded_void([&] {
            if (!THPDevice_Check(args[1])) throw Refused{"device: torch.device expected"};
            const c10::Device device = reinterpret_cast<THPDevice*>(args[1])->device;
            if (!device.is_cuda()) throw Refused{"device tensor expected"};
            index = c10::cuda::current_device();
            if (device.has_index() && device.index() != index)
                throw Refused{"tensor on cuda:" + std::to_string(device.index()) + ", but the current device is cuda:" + std::to_string(index)};
            stream = stream_of(args[0], index);
            cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
            const cudaError_t e = cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &status, &id);
            if (e != cudaSuccess) {
                (void)cudaGetLastError();
                throw std::runtime_error(cudaGetErrorString(e));
            }
            if (status != cudaStreamCaptureStatusActive) id = 0;
        }))
        return nullptr;
    return Py_BuildValue("(iKK)", index, (unsigned long long)(uintptr_t)stream, id);
}

// Sets what this thread may do while a stream is being captured (a
// cudaStreamCaptureMode); what it was.
PyObject* py_capture_mode(PyObject*, PyObject* const* args, Py_ssize_t n) {
    long long mode;
    if (!count(n, 1) || !number(args[0], &mode)) return nullptr;
    return guarded([&] {
        cudaStreamCaptureMode m = static_cast<cudaStreamCaptureMode>(mode);
        C10_CUDA_CHECK(cudaThreadExchangeStreamCaptureMode(&m));
        return static_cast<int>(m);
    });
}

PyMethodDef g_methods[] = {
    {"bind", py_bind, METH_VARARGS, "addresses of mq_linear_w4a16, mq_rope_kv_append, mq_kv_attention"},
    {"linear", reinterpret_cast<PyCFunction>(py_linear), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(py_append), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(py_attention), METH_FASTCALL, nullptr},
    {"place", reinterpret_cast<PyCFunction>(py_place), METH_FASTCALL, nullptr},
    {"capture_mode", reinterpret_cast<PyCFunction>(py_capture_mode), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_mq_torch", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__mq_torch(void) { return PyModule_Create(&g_module); }
