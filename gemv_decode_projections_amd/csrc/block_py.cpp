// Python entry points of the block operators' run functions (include/block.h):
// the checks of the tensors and the marshalling, compiled. A decode step makes
// these calls for a few microseconds of GPU work each, and the same checks in
// Python take longer than that (norm_run: 9.6 us a call, from here 4).
//
// Every function takes its tensors positionally, raises ValueError for a
// tensor that the operator does not take, and returns the library's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <string>
#include <vector>

#include "../../include/block.h"
#include "../../include/proj.h"

namespace {

// What block.py hands over: the C structure, and the GPU that its memory is on.
struct PyCache {
    blk_cache c;
    int device;
};
struct PyW4 {
    blk_w4 w;
    int device;
};
static_assert(offsetof(PyCache, device) == 64 && offsetof(PyW4, device) == 20, "block.py's _Cache and _W4");

struct Refused {
    std::string what;
};

void need(bool ok, const char *what)
{
    if (!ok)
        throw Refused{what};
}

std::string shape_text(const at::Tensor &t)
{
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i)
        s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        throw Refused{std::string(name) + " must be a tensor"};
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda())
        throw Refused{std::string(name) + " is on " + t.device().str() + ", not a GPU"};
    if (t.layout() != at::kStrided)
        throw Refused{std::string(name) + " must be a dense tensor"};
    return t;
}

int dtype_of(const at::Tensor &t)
{
    return t.scalar_type() == at::kBFloat16 ? BLK_BF16
           : t.scalar_type() == at::kHalf   ? BLK_F16
           : t.scalar_type() == at::kFloat  ? BLK_F32
                                            : -1;
}

void *pointer(const at::Tensor &t) { return t.data_ptr(); }

template <class T>
const T *address(PyObject *o)
{
    void *p = PyLong_AsVoidPtr(o);
    if (!p)
        throw Refused{"not an address"};
    return static_cast<const T *>(p);
}

at::Device gpu(int index) { return at::Device(at::kCUDA, (c10::DeviceIndex)index); }

// Launches go to the current device, whichever the stream's: it has to be the tensors'.
bool is_current(const at::Device &dev) { return c10::impl::VirtualGuardImpl(at::kCUDA).getDevice() == dev; }

void *raw(PyObject *o) { return PyLong_AsVoidPtr(o); }

// rows x width of one type and device, rows contiguous; returns the row stride.
int64_t rows_of(const at::Tensor &t, const char *name, int64_t rows, int64_t width, int dtype, const at::Device &dev)
{
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != width || dtype_of(t) != dtype || t.device() != dev ||
        (width > 1 && t.stride(1) != 1))
        throw Refused{std::string(name) + " has shape " + shape_text(t) + " of " + c10::toString(t.scalar_type()) +
                      ", expected contiguous rows " + std::to_string(rows) + " x " + std::to_string(width) + " of type " +
                      std::to_string(dtype) + " on " + dev.str()};
    return t.stride(0);
}

// A token-major tensor tokens x heads x dim of the cache's type.
void heads_of(const at::Tensor &t, const char *name, const blk_cache &c, int64_t tokens, int64_t heads,
              const at::Device &dev, int64_t &stride, int64_t &head_stride)
{
    if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != c.head_dim ||
        dtype_of(t) != c.dtype || t.device() != dev)
        throw Refused{std::string(name) + " has shape " + shape_text(t) + " of " + c10::toString(t.scalar_type()) +
                      ", expected " + std::to_string(tokens) + " x " + std::to_string(heads) + " x " +
                      std::to_string(c.head_dim) + " of the cache's type and device"};
    if (t.stride(2) != 1)
        throw Refused{std::string(name) + ": the elements of a head must be contiguous"};
    stride = t.stride(0);
    head_stride = t.stride(1);
}

blk_batch batch_of(PyObject *otable, PyObject *ostart, PyObject *olen, int64_t tokens, const at::Device &dev)
{
    const at::Tensor &table = tensor(otable, "table"), &start = tensor(ostart, "q_start"), &len = tensor(olen, "kv_len");
    for (const at::Tensor *t : {&table, &start, &len})
        need(t->scalar_type() == at::kInt && t->device() == dev, "table, q_start and kv_len must be int32 on the cache's device");
    need(table.dim() == 2 && start.dim() == 1 && len.dim() == 1, "table must have two dimensions, q_start and kv_len one");
    const int64_t seqs = table.size(0), width = table.size(1);
    if (start.size(0) != seqs + 1 || len.size(0) != seqs)
        throw Refused{std::to_string(seqs) + " table rows need " + std::to_string(seqs + 1) + " q_start and " +
                      std::to_string(seqs) + " kv_len entries, got " + std::to_string(start.size(0)) + " and " +
                      std::to_string(len.size(0))};
    need(width >= 1 && width <= INT32_MAX && seqs <= INT32_MAX && tokens <= INT32_MAX, "table has no columns, or too many");
    need((width == 1 || table.stride(1) == 1) && start.is_contiguous() && len.is_contiguous(),
         "q_start, kv_len and the rows of table must be contiguous");
    blk_batch b{};
    b.q_start = static_cast<const int32_t *>(pointer(start));
    b.kv_len = static_cast<const int32_t *>(pointer(len));
    b.table = static_cast<const int32_t *>(pointer(table));
    b.table_stride = seqs > 1 ? table.stride(0) : width;       // (one row's may be anything)
    b.table_width = (int)width;
    b.seqs = (int)seqs;
    b.tokens = (int)tokens;
    return b;
}

int int_of(PyObject *o, const char *name)
{
    const long v = PyLong_AsLong(o);
    if (PyErr_Occurred() || v < INT32_MIN || v > INT32_MAX) {
        PyErr_Clear();
        throw Refused{std::string(name) + " must be an integer of 32 bits"};
    }
    return (int)v;
}

double real_of(PyObject *o, const char *name)
{
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{std::string(name) + " must be a number"};
    }
    return v;
}

// The body of every entry: the number of arguments, no C++ exception past it.
template <class F>
PyObject *entry(Py_ssize_t got, Py_ssize_t want, F f)
{
    try {
        if (got != want) {
            PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
            return nullptr;
        }
        return PyLong_FromLong(f());
    } catch (const Refused &r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// attn_run(cache, workspace, workspace bytes, q, table, q_start, kv_len, out, gate, lse, max_q, scale, window, stream)
PyObject *attn_run(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return entry(n, 14, [&] {
        const PyCache &cache = *address<PyCache>(a[0]);
        const blk_cache &c = cache.c;
        const at::Tensor &q = tensor(a[3], "q"), &out = tensor(a[7], "out");
        need(q.dim() == 3, "q must be tokens x heads x head_dim");
        const int64_t tokens = q.size(0), heads = q.size(1);
        if (heads < 1 || heads % c.kv_heads)
            throw Refused{"q has " + std::to_string(heads) + " heads, the cache " + std::to_string(c.kv_heads)};
        const at::Device dev = gpu(cache.device);
        blk_attn_args x{};
        heads_of(q, "q", c, tokens, heads, dev, x.q_stride, x.q_head_stride);
        heads_of(out, "out", c, tokens, heads, dev, x.out_stride, x.out_head_stride);
        if (a[8] != Py_None) {
            const at::Tensor &gate = tensor(a[8], "gate");
            heads_of(gate, "gate", c, tokens, heads, dev, x.gate_stride, x.gate_head_stride);
            x.gate = pointer(gate);
        }
        if (a[9] != Py_None) {
            const at::Tensor &lse = tensor(a[9], "lse");
            need(lse.scalar_type() == at::kFloat && lse.dim() == 2 && lse.size(0) == tokens && lse.size(1) == heads &&
                     lse.is_contiguous() && lse.device() == dev,
                 "lse must be a contiguous float32 tensor tokens x heads on the cache's device");
            x.lse = static_cast<float *>(pointer(lse));
        }
        x.q = pointer(q);
        x.out = pointer(out);
        x.heads = (int)heads;
        x.max_q = a[10] == Py_None ? (int)std::max<int64_t>(std::min<int64_t>(tokens, INT32_MAX), 1) : int_of(a[10], "max_q");
        x.scale = a[11] == Py_None ? 1.0f / std::sqrt((float)c.head_dim) : (float)real_of(a[11], "scale");
        x.window = int_of(a[12], "window");
        const blk_batch b = batch_of(a[4], a[5], a[6], tokens, dev);
        if (!is_current(dev))
            return (int)PROJ_ERR_DEVICE;
        return blk_attn_run(&c, &b, &x, raw(a[1]), PyLong_AsSize_t(a[2]), raw(a[13]));
    });
}

// kv_append(cache, k, v, table, q_start, kv_len, stream)
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return entry(n, 7, [&] {
        const PyCache &cache = *address<PyCache>(a[0]);
        const blk_cache &c = cache.c;
        const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        need(k.dim() == 3, "k must be tokens x kv_heads x head_dim");
        const at::Device dev = gpu(cache.device);
        int64_t ks, kh, vs, vh;
        heads_of(k, "k", c, k.size(0), c.kv_heads, dev, ks, kh);
        heads_of(v, "v", c, k.size(0), c.kv_heads, dev, vs, vh);
        need((ks == vs || k.size(0) == 1) && (kh == vh || c.kv_heads == 1), "k and v have different strides");
        const blk_batch b = batch_of(a[3], a[4], a[5], k.size(0), dev);
        if (!is_current(dev))
            return (int)PROJ_ERR_DEVICE;
        return blk_kv_append(&c, &b, pointer(k), pointer(v), ks, kh, raw(a[6]));
    });
}

// kv_copy_pages(cache, src, dst, stream); src and dst sequences of integers
PyObject *kv_copy_pages(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return entry(n, 4, [&] {
        const PyCache &cache = *address<PyCache>(a[0]);
        const blk_cache &c = cache.c;
        std::vector<int32_t> pages[2];
        for (int i = 0; i < 2; ++i) {
            PyObject *seq = PySequence_Fast(a[1 + i], "");
            if (!seq) {
                PyErr_Clear();
                throw Refused{"src and dst must be sequences of page numbers"};
            }
            const Py_ssize_t m = PySequence_Fast_GET_SIZE(seq);
            PyObject **item = PySequence_Fast_ITEMS(seq);
            bool ok = true;
            pages[i].reserve(m);
            for (Py_ssize_t j = 0; j < m && ok; ++j) {
                const long p = PyLong_AsLong(item[j]);
                ok = !PyErr_Occurred() && p >= 0 && p <= INT32_MAX;
                pages[i].push_back((int32_t)p);
            }
            Py_DECREF(seq);
            PyErr_Clear();
            need(ok, "page numbers must be integers, not negative");
        }
        if (pages[0].size() != pages[1].size())
            throw Refused{std::to_string(pages[0].size()) + " source pages, " + std::to_string(pages[1].size()) + " destinations"};
        need(pages[0].size() <= INT32_MAX, "too many pages");
        if (!is_current(gpu(cache.device)))
            return (int)PROJ_ERR_DEVICE;
        return blk_kv_copy_pages(&c, pages[0].data(), pages[1].data(), (int)pages[0].size(), raw(a[3]));
    });
}

// w4_run(weight, packed, x, out, stream)
PyObject *w4_run(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return entry(n, 5, [&] {
        const PyW4 &weight = *address<PyW4>(a[0]);
        const blk_w4 &w = weight.w;
        const at::Device dev = gpu(weight.device);
        const at::Tensor &x = tensor(a[2], "x"), &out = tensor(a[3], "out");
        need(x.dim() == 2, "x must be m x k");
        const int64_t m = x.size(0), xs = rows_of(x, "x", m, w.k, w.dtype, dev);
        const int64_t os = rows_of(out, "out", m, w.n, w.dtype, dev);
        need(m <= INT32_MAX, "too many rows");
        if (!is_current(dev))
            return (int)PROJ_ERR_DEVICE;
        return blk_w4_run(&w, raw(a[1]), pointer(x), xs, (int)m, pointer(out), os, raw(a[4]));
    });
}

// norm_run(x, residual, out, weight_pre, weight_post, gate, alpha, eps, residual_out, stream)
PyObject *norm_run(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return entry(n, 10, [&] {
        const at::Tensor &out = tensor(a[2], "out"), &residual = tensor(a[1], "residual");
        need(out.dim() == 2, "out must be m x width");
        const at::Device dev = out.device();
        const int64_t m = out.size(0), width = out.size(1);
        const int type = dtype_of(out), rtype = dtype_of(residual);
        need(type == BLK_BF16 || type == BLK_F16, "out must be bfloat16 or float16");
        need(rtype == type || rtype == BLK_F32, "residual must be of out's type or float32");
        need(m <= INT32_MAX && width <= INT32_MAX, "too many rows or columns");
        auto vector = [&](PyObject *o, const char *name) -> const void * {
            const at::Tensor &t = tensor(o, name);
            if (t.dim() != 1 || t.size(0) != width || dtype_of(t) != type || t.device() != dev || (width > 1 && t.stride(0) != 1))
                throw Refused{std::string(name) + " has shape " + shape_text(t) + ", expected a contiguous vector of " +
                              std::to_string(width) + " of out's type and device"};
            return pointer(t);
        };
        blk_norm_args x{};
        x.width = (int)width;
        x.dtype = type;
        x.residual_dtype = rtype;
        x.alpha = (float)real_of(a[6], "alpha");
        x.eps = (float)real_of(a[7], "eps");
        x.out = pointer(out);
        x.out_stride = rows_of(out, "out", m, width, type, dev);
        x.residual = pointer(residual);
        x.residual_stride = rows_of(residual, "residual", m, width, rtype, dev);
        need(a[3] != Py_None, "weight_pre is needed");
        x.weight_pre = vector(a[3], "weight_pre");
        if (a[0] == Py_None) {
            need(a[4] == Py_None && a[5] == Py_None && a[8] == Py_None, "weight_post, gate and residual_out need x");
        } else {
            const at::Tensor &in = tensor(a[0], "x"), &ro = a[8] == Py_None ? residual : tensor(a[8], "residual_out");
            x.x = pointer(in);
            x.x_stride = rows_of(in, "x", m, width, type, dev);
            x.residual_out = pointer(ro);
            x.residual_out_stride = rows_of(ro, "residual_out", m, width, rtype, dev);
            if (a[4] != Py_None)
                x.weight_post = vector(a[4], "weight_post");
            if (a[5] != Py_None) {
                const at::Tensor &gate = tensor(a[5], "gate");
                if (gate.dim() == 1) {
                    x.gate = vector(a[5], "gate");
                } else {
                    x.gate = pointer(gate);
                    x.gate_stride = rows_of(gate, "gate", m, width, type, dev);
                }
            }
        }
        if (!is_current(dev))
            return (int)PROJ_ERR_DEVICE;
        return blk_norm_run(&x, (int)m, raw(a[9]));
    });
}

PyMethodDef methods[] = {
    {"attn_run", (PyCFunction)(void (*)(void))attn_run, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, nullptr},
    {"kv_copy_pages", (PyCFunction)(void (*)(void))kv_copy_pages, METH_FASTCALL, nullptr},
    {"w4_run", (PyCFunction)(void (*)(void))w4_run, METH_FASTCALL, nullptr},
    {"norm_run", (PyCFunction)(void (*)(void))norm_run, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
