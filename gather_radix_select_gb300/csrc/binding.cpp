// binding.cpp -- the Python module _binding: the entry points of include/sel/cache_serving.h on torch tensors.
// Argument checks on tensors and marshalling only; what is computed runs in libsel.so's kernels.
//
// The calls of a serving step are short on the GPU (a token appended to each of 32 sequences: 3 us), and by way of
// ctypes the host took longer than that to make them: 20 us for the append with queries, 28 us for an attention in
// two launches; from here 5.5 and 13.  So these have a module of their own.  It uses whichever build of the library
// was loaded (bind).
#include <Python.h>

#include <cmath>
#include <type_traits>

#include <dlfcn.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/sel/cache_serving.h"

namespace {

struct Library {
    decltype(&sel_cache_append) append;
    decltype(&sel_cache_attention_window) window;
    decltype(&sel_cache_attention_window_workspace_size) window_size;
    decltype(&sel_cache_attention_shared) shared;
    decltype(&sel_cache_attention_shared_workspace_size) shared_size;
} lib;

// What is wrong with the arguments: a ValueError.
struct Refused {
    const char *why;
};
void require(bool ok, const char *why)
{
    if (!ok) throw Refused{why};
}

const at::Tensor *tensor(PyObject *o, const char *why)  // null: None
{
    if (o == Py_None) return nullptr;
    require(THPVariable_Check(o), why);
    return &THPVariable_Unpack(o);
}
const at::Tensor &given(PyObject *o, const char *why)
{
    require(o != Py_None && THPVariable_Check(o), why);
    return THPVariable_Unpack(o);
}

// A Python error has been set.
struct Raised {};
int64_t integer(PyObject *o)
{
    PyObject *n = PyNumber_Long(o);
    if (!n) throw Raised{};
    const long long v = PyLong_AsLongLong(n);
    Py_DECREF(n);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

int type_of_rows(const at::Tensor &t)
{
    return t.scalar_type() == at::kFloat ? SEL_F32 : t.scalar_type() == at::kBFloat16 ? SEL_BF16 : -1;
}
int type_of_index(const at::Tensor &t)
{
    return t.scalar_type() == at::kInt ? SEL_I32 : t.scalar_type() == at::kLong ? SEL_I64 : -1;
}

sel_cache cache_of(const at::Tensor &cache, const at::Tensor *scales)
{
    const bool codes = cache.scalar_type() == at::kFloat8_e4m3fn;
    require((codes || cache.scalar_type() == at::kBFloat16) && cache.dim() == 3,
            "cache must be a 3-D bfloat16 or float8_e4m3fn tensor [pages, page_size, d]");
    require(cache.is_cuda(), "cache must be a CUDA tensor");
    sel_cache c{};
    c.data = cache.data_ptr();
    c.dtype = codes ? int{SEL_E4M3} : int{SEL_BF16};
    c.pages = cache.size(0), c.page_size = cache.size(1), c.d = cache.size(2);
    require(c.d <= 1 || cache.stride(2) == 1, "cache rows must be contiguous in their last dimension");
    c.row_stride = c.page_size == 1 ? c.d : cache.stride(1);
    c.page_stride = c.pages == 1 ? c.page_size * c.row_stride : cache.stride(0);
    if (!codes) {
        require(!scales, "a bfloat16 cache has no scales");
        return c;
    }
    const int64_t runs = (c.d + SEL_CACHE_GROUP - 1) / SEL_CACHE_GROUP;
    require(scales && scales->scalar_type() == at::kFloat && scales->dim() == 3 && scales->size(0) == c.pages &&
                scales->size(1) == c.page_size && scales->size(2) == runs && scales->device() == cache.device(),
            "a float8_e4m3fn cache needs float32 scales [pages, page_size, ceil(d / 128)] on its device");
    require(runs <= 1 || scales->stride(2) == 1, "scales must be contiguous in their last dimension");
    c.scales = scales->data_ptr<float>();
    c.scale_row_stride = c.page_size == 1 ? runs : scales->stride(1);
    c.scale_page_stride = c.pages == 1 ? c.page_size * c.scale_row_stride : scales->stride(0);
    return c;
}

struct Table {
    const int32_t *data;
    int64_t b, max_pages, stride;
};
Table table_of(const at::Tensor &t, at::Device dev)
{
    require(t.scalar_type() == at::kInt && t.dim() == 2 && t.device() == dev,
            "page_table must be an int32 tensor [b, max_pages] on the cache's device");
    require(t.size(0) >= 1, "page_table needs a row for each sequence");
    require(t.size(1) <= 1 || t.stride(1) == 1, "page_table rows must be contiguous");
    return Table{t.data_ptr<int32_t>(), t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : t.size(1)};
}

int32_t *flag_of(const at::Tensor *t, at::Device dev)
{
    if (!t) return nullptr;
    require(t->scalar_type() == at::kInt && t->numel() >= 1 && t->device() == dev,
            "err_flag must be an int32 tensor on the cache's device");
    return t->data_ptr<int32_t>();
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, at::Device dev)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// (x, cache, page_table, positions, rotation, scales, first, interleaved, q, q_out, err_flag) -> q_out, None, or a status
PyObject *append(PyObject *const *args)
{
    const at::Tensor &cache = given(args[1], "cache must be a 3-D bfloat16 or float8_e4m3fn tensor [pages, page_size, d]");
    const sel_cache c = cache_of(cache, tensor(args[5], "scales must be a tensor"));
    const at::Device dev = cache.device();
    const char *of_x = "x must be a bfloat16 or float32 tensor [tokens, d] on the cache's device";
    const at::Tensor &x = given(args[0], of_x);
    const int x_type = type_of_rows(x);
    require(x_type >= 0 && x.dim() == 2 && x.device() == dev && x.size(1) == c.d, of_x);
    const int64_t tokens = x.size(0), d = c.d;
    require(d <= 1 || x.stride(1) == 1, "rows of x must be contiguous");
    const Table t = table_of(given(args[2], "page_table must be a tensor"), dev);
    const char *of_positions = "positions must be a contiguous int32/int64 tensor with one entry per token";
    const at::Tensor &positions = given(args[3], of_positions);
    const int pos_type = type_of_index(positions);
    require(pos_type >= 0 && positions.dim() == 1 && positions.size(0) == tokens && positions.device() == dev &&
                positions.is_contiguous(),
            of_positions);
    const char *of_rotation = "rotation must be a float32 tensor [positions, rot] on the cache's device";
    const at::Tensor &rotation = given(args[4], of_rotation);
    require(rotation.scalar_type() == at::kFloat && rotation.dim() == 2 && rotation.device() == dev, of_rotation);
    const int64_t known = rotation.size(0), rot = rotation.size(1);
    require(rot <= 1 || rotation.stride(1) == 1, "rows of rotation must be contiguous");
    sel_rotation turn{};
    turn.table = rotation.data_ptr<float>();
    turn.positions = known;
    turn.stride = known > 1 ? rotation.stride(0) : rot;
    turn.first = args[6] == Py_None ? d - rot : integer(args[6]);
    turn.rot = rot;
    turn.interleaved = truth(args[7]);
    const at::Tensor *q = tensor(args[8], "q must be a tensor"), *q_out = tensor(args[9], "q_out must be a tensor");
    int q_type = 0;
    int64_t h = 0, q_row = 0, q_head = 0;
    const void *q_ptr = nullptr;
    if (q) {
        q_type = type_of_rows(*q);
        require(q_type >= 0 && q->dim() == 3 && q->device() == dev && q->size(0) == tokens && q->size(2) == d,
                "q must be a bfloat16 or float32 tensor [tokens, h, d] on the cache's device");
        h = q->size(1);
        require(d <= 1 || q->stride(2) == 1, "q must be contiguous in its last dimension");
        q_row = tokens > 1 ? q->stride(0) : h * d;
        q_head = h > 1 ? q->stride(1) : d;
        q_ptr = tokens > 0 ? q->data_ptr() : x.data_ptr();
    }
    require(!q_out || (q && q_out->sizes() == q->sizes() && q_out->is_contiguous() &&
                       q_out->scalar_type() == at::kBFloat16 && q_out->device() == dev),
            "q_out must be a contiguous bf16 tensor of q's shape");
    int32_t *err = flag_of(tensor(args[10], "err_flag must be a tensor"), dev);

    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor to;
    if (q) to = q_out ? *q_out : make({tokens, h, d}, at::kBFloat16, dev);
    void *out = q ? to.data_ptr() : nullptr;
    void *stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = lib.append(x.data_ptr(), x_type, tokens, tokens > 1 ? x.stride(0) : d, &c, t.data, t.b, t.max_pages, t.stride,
                        positions.data_ptr(), pos_type, &turn, q_ptr, q_type, h, q_row, q_head, out, err, stream);
    Py_END_ALLOW_THREADS
    if (status != SEL_OK) return PyLong_FromLong(status);
    if (!q) Py_RETURN_NONE;
    if (q_out) return Py_NewRef(args[9]);
    return THPVariable_Wrap(std::move(to));
}

// (q, cache, page_table, scales, end, dv, scale, return_lse, out, err_flag, window, sinks, shared; window None: shared)
// -> (out, lse or None), or a status
PyObject *attention(PyObject *const *args)
{
    const at::Tensor &cache = given(args[1], "cache must be a 3-D bfloat16 or float8_e4m3fn tensor [pages, page_size, d]");
    const sel_cache c = cache_of(cache, tensor(args[3], "scales must be a tensor"));
    const at::Device dev = cache.device();
    const Table t = table_of(given(args[2], "page_table must be a tensor"), dev);
    const char *of_q = "q must be a bfloat16 tensor [rows, h, d] on the cache's device";
    const at::Tensor &q = given(args[0], of_q);
    const int64_t d = c.d;
    require(q.scalar_type() == at::kBFloat16 && q.dim() == 3 && q.device() == dev && q.size(2) == d, of_q);
    const int64_t rows = q.size(0), h = q.size(1);
    require(d <= 1 || q.stride(2) == 1, "q must be contiguous in its last dimension");
    const at::Tensor *end = tensor(args[4], "end must be a tensor");
    require(!end || (end->scalar_type() == at::kInt && end->dim() == 1 && end->size(0) == rows && end->device() == dev &&
                     end->is_contiguous()),
            "end must be a contiguous int32 tensor with one entry per row");
    const int64_t dv = args[5] == Py_None ? d : integer(args[5]);
    double scale = d > 0 ? 1.0 / std::sqrt(static_cast<double>(d)) : 1.0;
    if (args[6] != Py_None) {
        scale = PyFloat_AsDouble(args[6]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    }
    const bool return_lse = truth(args[7]);
    const at::Tensor *out = tensor(args[8], "out must be a tensor");
    require(!out || (out->dim() == 3 && out->size(0) == rows && out->size(1) == h && out->size(2) == dv &&
                     out->is_contiguous() && out->scalar_type() == at::kBFloat16 && out->device() == dev),
            "out must be a contiguous bf16 [rows, h, dv] tensor");
    int32_t *err = flag_of(tensor(args[9], "err_flag must be a tensor"), dev);
    const bool window = args[10] != Py_None;
    const int64_t limit = integer(args[window ? 10 : 12]), sinks = window ? integer(args[11]) : 0;

    const c10::cuda::CUDAGuard guard(dev);
    const at::Tensor to = out ? *out : make({rows, h, dv < 0 ? 0 : dv}, at::kBFloat16, dev);
    at::Tensor lse, ws;
    if (return_lse) lse = make({rows, h}, at::kFloat, dev);
    // Scratch of the call's own, from the stream's pool: two launches pass data through it, and another thread's call
    // on the same stream may come between them.
    const size_t need = window ? lib.window_size(rows, h, d, dv, t.b, t.max_pages, c.page_size, limit, sinks)
                               : lib.shared_size(rows, h, d, dv, t.b, t.max_pages, c.page_size, limit);
    if (need > 0) ws = make({static_cast<int64_t>(need)}, at::kByte, dev);
    void *stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    const int32_t *ends = end ? end->data_ptr<int32_t>() : nullptr;
    float *sums = return_lse ? lse.data_ptr<float>() : nullptr;
    void *scratch = need > 0 ? ws.data_ptr() : nullptr;
    const int64_t q_row = rows > 1 ? q.stride(0) : h * d, q_head = h > 1 ? q.stride(1) : d;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = window ? lib.window(q.data_ptr(), rows, h, q_row, q_head, &c, t.data, t.b, t.max_pages, t.stride, ends, limit,
                                 sinks, dv, static_cast<float>(scale), to.data_ptr(), sums, scratch, need, err, stream)
                    : lib.shared(q.data_ptr(), rows, h, q_row, q_head, &c, t.data, t.b, t.max_pages, t.stride, ends, limit,
                                 dv, static_cast<float>(scale), to.data_ptr(), sums, scratch, need, err, stream);
    Py_END_ALLOW_THREADS
    if (status != SEL_OK) return PyLong_FromLong(status);
    PyObject *pair = PyTuple_New(2);
    if (!pair) throw Raised{};
    PyTuple_SET_ITEM(pair, 0, out ? Py_NewRef(args[8]) : THPVariable_Wrap(to));
    PyTuple_SET_ITEM(pair, 1, return_lse ? THPVariable_Wrap(std::move(lse)) : Py_NewRef(Py_None));
    if (!PyTuple_GET_ITEM(pair, 0) || !PyTuple_GET_ITEM(pair, 1)) {
        Py_DECREF(pair);
        throw Raised{};
    }
    return pair;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
        return nullptr;
    }
    try {
        if (!lib.append) throw Refused{"the library is not bound"};
        return F(args);
    } catch (const Refused &r) {
        PyErr_SetString(PyExc_ValueError, r.why);
    } catch (const Raised &) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// (handle of the loaded library)
PyObject *bind(PyObject *, PyObject *handle)
{
    void *from = PyLong_AsVoidPtr(handle);
    if (!from && PyErr_Occurred()) return nullptr;
    Library found{};
    auto find = [&](auto &f, const char *name) {
        f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(from, name));
        if (!f) PyErr_Format(PyExc_RuntimeError, "%s is not in the library", name);
        return f != nullptr;
    };
    if (!find(found.append, "sel_cache_append") || !find(found.window, "sel_cache_attention_window") ||
        !find(found.window_size, "sel_cache_attention_window_workspace_size") ||
        !find(found.shared, "sel_cache_attention_shared") ||
        !find(found.shared_size, "sel_cache_attention_shared_workspace_size"))
        return nullptr;
    lib = found;
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyCFunction fast()
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(static_cast<_PyCFunctionFast>(entry<F, N>)));
}

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"cache_append", fast<append, 11>(), METH_FASTCALL, nullptr},
                         {"cache_attention", fast<attention, 13>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
