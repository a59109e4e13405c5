// pkv_torch.cc -- the calls that a decode step makes in every layer, from torch
// tensors to the C ABI: the binding's checks of types, places and shapes in C++.
// A call of 20 tensors takes 12 us of host time when they are checked and
// converted in Python, several times what its kernel takes for a few tokens.
//
// The functions take their arguments by place, as the Python binding passes them
// on, and return a pkv_status.  A wrong tensor raises ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "pkv.h"

namespace {

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonError {}; // the Python error is set

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kI64 = at::kLong, kU8 = at::kByte;

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        throw Refused(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}

// The device a call runs on: its first tensor's, which has to be the current
// one (the library launches on the current device).
int device_of(PyObject *o, const char *name)
{
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda())
        throw Refused(std::string(name) + ": expected a CUDA tensor");
    const int dev = t.get_device();
    if (dev != c10::cuda::current_device())
        throw Refused(std::string(name) + " is on cuda:" + std::to_string(dev) + ", which is not the current device");
    return dev;
}

void *stream_of(int dev)
{
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
}

void *check(const at::Tensor &t, int dev, const char *name, at::ScalarType type)
{
    if (t.scalar_type() != type || !t.is_contiguous() || !t.is_cuda() || t.get_device() != dev)
        throw Refused(std::string(name) + ": expected a contiguous " + c10::toString(type) + " tensor on cuda:" +
                      std::to_string(dev));
    return t.data_ptr();
}

// Address of a contiguous tensor of this type and shape on this device; NULL for None.
void *at_(PyObject *o, int dev, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape)
{
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = tensor(o, name);
    void *p = check(t, dev, name, type);
    if (t.sizes() != c10::IntArrayRef(shape)) {
        std::string want, got;
        for (int64_t n : shape)
            want += " " + std::to_string(n);
        for (int64_t n : t.sizes())
            got += " " + std::to_string(n);
        throw Refused(std::string(name) + ": expected shape" + want + ", got" + got);
    }
    return p;
}
// The same, of any shape.
void *any_at(PyObject *o, int dev, const char *name, at::ScalarType type)
{
    return o == Py_None ? nullptr : check(tensor(o, name), dev, name, type);
}
template <typename T> T *as(void *p)
{
    return static_cast<T *>(p);
}

c10::IntArrayRef sizes(PyObject *o, const char *name, size_t dims)
{
    const at::Tensor &t = tensor(o, name);
    if ((size_t)t.dim() != dims)
        throw Refused(std::string(name) + ": expected " + std::to_string(dims) + " dimensions");
    return t.sizes();
}

int32_t narrow(int64_t x)
{
    if (x < INT32_MIN || x > INT32_MAX)
        throw Refused("a number does not fit in 32 bits");
    return (int32_t)x;
}
int32_t whole(PyObject *o)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred())
        throw PythonError();
    return narrow(x);
}
float real(PyObject *o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred())
        throw PythonError();
    return (float)x;
}

pkv_cache_desc desc_of(PyObject *k_cache, int32_t layout)
{
    const c10::IntArrayRef s = sizes(k_cache, "k_cache", 4);
    const bool nhd = layout == PKV_NHD;
    return {narrow(s[0]), narrow(s[nhd ? 1 : 2]), narrow(s[nhd ? 2 : 1]), narrow(s[3]), layout};
}

// Runs f and turns what it throws into a Python error.
template <typename F> PyObject *call(const char *name, Py_ssize_t n, Py_ssize_t want, F f)
{
    try {
        if (n != want)
            throw Refused(std::string(name) + ": wrong number of arguments");
        return PyLong_FromLong(f());
    } catch (const PythonError &) {
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, name);
    }
    return nullptr;
}

// q, k, positions, freqs, pairing, attn_factor, q_out, k_out
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call("rope", n, 8, [&] {
        PyObject *some = a[0] != Py_None ? a[0] : a[1];
        const int dev = device_of(some, a[0] != Py_None ? "q" : "k");
        const c10::IntArrayRef s = sizes(some, "q or k", 3);
        const int64_t T = s[0], D = s[2];
        const int64_t Hq = a[0] != Py_None ? sizes(a[0], "q", 3)[1] : 0, Hk = a[1] != Py_None ? sizes(a[1], "k", 3)[1] : 0;
        const void *freqs = any_at(a[3], dev, "freqs", kI64);
        return pkv_rope(at_(a[0], dev, "q", kBf16, {T, Hq, D}), at_(a[1], dev, "k", kBf16, {T, Hk, D}),
                        as<int32_t>(at_(a[2], dev, "positions", kI32, {T})), narrow(T), narrow(Hq), narrow(Hk), narrow(D),
                        static_cast<const uint64_t *>(freqs), narrow(2 * tensor(a[3], "freqs").numel()), whole(a[4]),
                        real(a[5]), at_(a[6], dev, "q_out", kBf16, {T, Hq, D}), at_(a[7], dev, "k_out", kBf16, {T, Hk, D}),
                        stream_of(dev));
    });
}

// k_cache, v_cache, q, k_new, v_new, block_table, cache_seqlens, freqs, pairing, attn_factor, append_indptr, positions,
// evicted, q_out, err_flag, layout
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call("rope_append", n, 16, [&] {
        const int dev = device_of(a[3], "k_new");
        const pkv_cache_desc d = desc_of(a[0], whole(a[15]));
        const c10::IntArrayRef pool = tensor(a[0], "k_cache").sizes();
        const int64_t T = sizes(a[3], "k_new", 3)[0], B = sizes(a[6], "cache_seqlens", 1)[0];
        const int64_t width = sizes(a[5], "block_table", 2)[1], K = d.num_kv_heads, D = d.head_dim;
        const int64_t Hq = a[2] != Py_None ? sizes(a[2], "q", 3)[1] : 0;
        const void *freqs = any_at(a[7], dev, "freqs", kI64);
        return pkv_rope_append(
            &d, any_at(a[0], dev, "k_cache", kBf16), at_(a[1], dev, "v_cache", kBf16, {pool[0], pool[1], pool[2], pool[3]}),
            at_(a[2], dev, "q", kBf16, {T, Hq, D}), at_(a[3], dev, "k_new", kBf16, {T, K, D}),
            at_(a[4], dev, "v_new", kBf16, {T, K, D}), narrow(T), as<int32_t>(at_(a[10], dev, "append_indptr", kI32, {B + 1})),
            as<int32_t>(at_(a[11], dev, "positions", kI32, {T})), as<int32_t>(at_(a[12], dev, "evicted", kI32, {B})),
            static_cast<const uint64_t *>(freqs), narrow(2 * tensor(a[7], "freqs").numel()), whole(a[8]), real(a[9]),
            as<int32_t>(at_(a[5], dev, "block_table", kI32, {B, width})), narrow(width),
            as<int32_t>(at_(a[6], dev, "cache_seqlens", kI32, {B})), narrow(B), narrow(Hq),
            at_(a[13], dev, "q_out", kBf16, {T, Hq, D}), as<int32_t>(any_at(a[14], dev, "err_flag", kI32)), stream_of(dev));
    });
}

// k_cache, q, lse, block_table, cache_seqlens, softmax_scale, mass, qo_indptr, fresh_from, evicted, slot_pos, workspace,
// err_flag, layout
PyObject *attn_mass(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call("attn_mass", n, 14, [&] {
        const int dev = device_of(a[1], "q");
        const pkv_cache_desc d = desc_of(a[0], whole(a[13]));
        const c10::IntArrayRef q = sizes(a[1], "q", 3), table = sizes(a[3], "block_table", 2);
        const int64_t T = q[0], Hq = q[1], B = table[0], width = table[1], K = d.num_kv_heads;
        const int64_t slots = sizes(a[6], "mass", 3)[2];
        return pkv_attn_mass(
            &d, any_at(a[0], dev, "k_cache", kBf16), at_(a[1], dev, "q", kBf16, {T, Hq, d.head_dim}),
            as<int32_t>(at_(a[7], dev, "qo_indptr", kI32, {B + 1})), as<float>(at_(a[2], dev, "lse", kF32, {T, Hq})),
            as<int32_t>(any_at(a[3], dev, "block_table", kI32)), narrow(width),
            as<int32_t>(at_(a[4], dev, "cache_seqlens", kI32, {B})), narrow(B), narrow(Hq), narrow(T), real(a[5]),
            as<int32_t>(at_(a[8], dev, "fresh_from", kI32, {B})), as<int32_t>(at_(a[9], dev, "evicted", kI32, {B})),
            as<float>(at_(a[6], dev, "mass", kF32, {B, K, slots})), as<int32_t>(at_(a[10], dev, "slot_pos", kI32, {B, K, slots})),
            narrow(slots), any_at(a[11], dev, "workspace", kU8), (size_t)tensor(a[11], "workspace").numel(),
            as<int32_t>(any_at(a[12], dev, "err_flag", kI32)), stream_of(dev));
    });
}

// mass, slot_pos, cache_seqlens, evicted, budgets, sink, recent, moves, num_moves, row_lens, err_flag
PyObject *evict_plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call("evict_plan", n, 11, [&] {
        const int dev = device_of(a[0], "mass");
        const c10::IntArrayRef s = sizes(a[0], "mass", 4);
        const int64_t layers = s[0], B = s[1], K = s[2], slots = s[3], most = sizes(a[7], "moves", 5)[3];
        return pkv_evict_plan(
            as<float>(any_at(a[0], dev, "mass", kF32)), as<int32_t>(at_(a[1], dev, "slot_pos", kI32, {layers, B, K, slots})),
            narrow(layers), narrow(B), narrow(K), narrow(slots), as<int32_t>(at_(a[2], dev, "cache_seqlens", kI32, {B})),
            as<int32_t>(at_(a[3], dev, "evicted", kI32, {B})), as<int32_t>(at_(a[4], dev, "budgets", kI32, {B})), whole(a[5]),
            whole(a[6]), as<int32_t>(at_(a[7], dev, "moves", kI32, {layers, B, K, most, 2})), narrow(most),
            as<int32_t>(at_(a[8], dev, "num_moves", kI32, {layers, B, K})), as<int32_t>(at_(a[9], dev, "row_lens", kI32, {B, 2})),
            as<int32_t>(any_at(a[10], dev, "err_flag", kI32)), stream_of(dev));
    });
}

// (address of the pools' descriptor, addresses of the two pointer arrays, layers, kv heads, device), moves, num_moves,
// row_lens, block_table, cache_seqlens, evicted, mass, slot_pos, err_flag
PyObject *evict_apply(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call("evict_apply", n, 15, [&] {
        const auto *d = static_cast<const pkv_cache_desc *>(PyLong_AsVoidPtr(a[0]));
        auto *k = static_cast<void *const *>(PyLong_AsVoidPtr(a[1])), *v = static_cast<void *const *>(PyLong_AsVoidPtr(a[2]));
        if (PyErr_Occurred())
            throw PythonError();
        const int64_t layers = whole(a[3]), K = whole(a[4]);
        const int dev = device_of(a[6], "moves");
        if (dev != whole(a[5]))
            throw Refused("moves and caches on different devices");
        const c10::IntArrayRef table = sizes(a[9], "block_table", 2);
        const int64_t B = table[0], width = table[1], most = sizes(a[6], "moves", 5)[3];
        PyObject *state = a[12] != Py_None ? a[12] : a[13];
        const int64_t slots = state != Py_None ? sizes(state, "mass or slot_pos", 4)[3] : 1;
        return pkv_evict_apply(
            d, narrow(layers), k, v, as<int32_t>(at_(a[6], dev, "moves", kI32, {layers, B, K, most, 2})), narrow(most),
            as<int32_t>(at_(a[7], dev, "num_moves", kI32, {layers, B, K})), as<int32_t>(at_(a[8], dev, "row_lens", kI32, {B, 2})),
            as<int32_t>(any_at(a[9], dev, "block_table", kI32)), narrow(width),
            as<float>(at_(a[12], dev, "mass", kF32, {layers, B, K, slots})),
            as<int32_t>(at_(a[13], dev, "slot_pos", kI32, {layers, B, K, slots})), narrow(slots),
            as<int32_t>(at_(a[10], dev, "cache_seqlens", kI32, {B})), as<int32_t>(at_(a[11], dev, "evicted", kI32, {B})),
            narrow(B), as<int32_t>(any_at(a[14], dev, "err_flag", kI32)), stream_of(dev));
    });
}

#define PKV_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {PKV_METHOD(rope),       PKV_METHOD(rope_append), PKV_METHOD(attn_mass),
                          PKV_METHOD(evict_plan), PKV_METHOD(evict_apply), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "pkv_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit_pkv_torch(void)
{
    return PyModule_Create(&kModule);
}
