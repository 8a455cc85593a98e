// paged_binding.cpp -- the Python side of the paged key-value cache's entry points: checks of the
// tensors, allocation of outputs and workspaces, and the call of the C ABI on the current stream.
//
// A decode step makes these calls once a layer on inputs that the GPU is done with in microseconds,
// so the time to get from Python to the launch counts: read off in C++ from the tensor objects,
// shapes, strides, pointers and the stream cost well under a microsecond a call, where Python and
// ctypes take 9 to 10.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>

#include "gret.h"

namespace {

PyObject* check_status = nullptr;      // raises for a status that is not GRET_OK

struct Refused {};                     // a Python error is set

template <typename... Args>
[[noreturn]] void refuse(PyObject* type, const char* format, Args... args) {
    PyErr_Format(type, format, args...);
    throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

const at::Tensor* optional(PyObject* o, const char* name) {
    return o == Py_None ? nullptr : &tensor(o, name);
}

int to_int(int64_t x, const char* name) {
    if (x < INT_MIN || x > INT_MAX) refuse(PyExc_ValueError, "%s is out of range", name);
    return (int)x;
}

int to_int(PyObject* o, const char* name) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Refused{};
    return to_int((int64_t)x, name);
}

bool to_bool(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Refused{};
    return x;
}

// The device and the stream of a call: every tensor is on that device, a GPU; while this lives,
// both are current.  `stream` is a torch stream, or None for the current one.
struct Scope {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard stream;
    gret_stream_t raw;

    Scope(PyObject* given, const at::Tensor& first,
          std::initializer_list<const at::Tensor*> others) {
        if (!first.is_cuda()) refuse(PyExc_ValueError, "paged cache tensors must be on a GPU");
        for (const at::Tensor* t : others)
            if (t && t->device() != first.device())
                refuse(PyExc_ValueError, "paged cache tensors must be on one device");
        if (given == Py_None) {
            device.set_device(first.device());
        } else {
            if (!THPStream_Check(given)) refuse(PyExc_TypeError, "stream must be a torch stream");
            const THPStream* s = reinterpret_cast<THPStream*>(given);
            if ((c10::DeviceType)s->device_type != first.device().type() ||
                s->device_index != first.device().index())
                refuse(PyExc_ValueError, "stream must be of the tensors' device");
            stream.reset_stream(c10::Stream::unpack3(
                s->stream_id, (c10::DeviceIndex)s->device_index, (c10::DeviceType)s->device_type));
        }
        raw = (gret_stream_t)c10::cuda::getCurrentCUDAStream(first.device().index()).stream();
    }
};

// An int32 argument's pointer (no argument: NULL).
int32_t* int32s(const at::Tensor* t, const char* name, int64_t n) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
        refuse(PyExc_ValueError, "%s must be contiguous int32 [%lld]", name, (long long)n);
    return static_cast<int32_t*>(t->data_ptr());
}

struct Table {
    int32_t* entries;
    int64_t stride;
    int max_pages;

    Table(const at::Tensor& t, int64_t rows) {
        if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != rows ||
            (t.size(1) > 1 && rows && t.stride(1) != 1))
            refuse(PyExc_ValueError,
                   "page_table must be int32 [%lld, max_pages] with contiguous rows",
                   (long long)rows);
        entries = static_cast<int32_t*>(t.data_ptr());
        max_pages = to_int(t.size(1), "max_pages");
        stride = rows > 1 ? t.stride(0) : max_pages;
    }
};

gret_dtype_t dtype_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return GRET_BF16;
    if (t.scalar_type() != at::kFloat)
        refuse(PyExc_TypeError, "q/k/v must be bfloat16 or float32, got %s",
               c10::toString(t.scalar_type()));
    return GRET_F32;
}

struct Pool {
    void *k, *v;
    int64_t sp, st, sh;
    int n_pages, page, H, d;
    gret_dtype_t dtype;

    Pool(const at::Tensor& kp, const at::Tensor& vp, bool head_major) {
        if (kp.dim() != 4 || kp.sizes() != vp.sizes() || kp.scalar_type() != vp.scalar_type())
            refuse(PyExc_ValueError, "k_pages and v_pages must be 4-D and alike");
        if (kp.strides() != vp.strides() || kp.stride(3) != 1)
            refuse(PyExc_ValueError, "k_pages and v_pages must share strides, the last one 1");
        const int tok = head_major ? 2 : 1, head = head_major ? 1 : 2;
        dtype = dtype_of(kp);
        k = kp.data_ptr();
        v = vp.data_ptr();
        sp = kp.stride(0);
        st = kp.stride(tok);
        sh = kp.stride(head);
        n_pages = to_int(kp.size(0), "pages");
        page = to_int(kp.size(tok), "page size");
        H = to_int(kp.size(head), "heads");
        d = to_int(kp.size(3), "d");
    }
};

// A given workspace, or one of the call's own: memory of torch's allocator for the current stream,
// without a tensor around it.
struct Workspace {
    c10::DataPtr own;
    void* at;
    size_t bytes;

    Workspace(const at::Tensor* given, size_t need) {
        if (given) {
            if (!given->is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
            at = given->data_ptr();
            bytes = given->nbytes();
        } else {
            bytes = need > 16 ? need : 16;
            own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
            at = own.get();
        }
    }
};

at::Tensor int32_output(const at::Tensor* given, int64_t n, const at::Tensor& like) {
    return given ? *given : at::empty({n}, like.options().dtype(at::kInt));
}

void check(const char* fn, gret_status_t status) {
    if (status == GRET_OK) return;
    PyObject* r = PyObject_CallFunction(check_status, "si", fn, (int)status);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s failed", fn);
    throw Refused{};
}

// (q, seq_lens, page_table, k_pages, v_pages, window, scale, head_major, o, lse, status, workspace,
// stream)
PyObject* attention_decode(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &lens = tensor(a[1], "seq_lens"),
                     &pt = tensor(a[2], "page_table"), &kp = tensor(a[3], "k_pages"),
                     &vp = tensor(a[4], "v_pages");
    const int window = to_int(a[5], "window");
    const at::Tensor *given_o = optional(a[8], "o"),
                     *given_lse = a[9] == Py_True ? nullptr : optional(a[9], "lse"),
                     *status = optional(a[10], "status"), *ws = optional(a[11], "workspace");
    const Pool p(kp, vp, to_bool(a[7]));
    if (q.dim() != 3 || q.size(2) != p.d || q.scalar_type() != kp.scalar_type() ||
        !q.is_contiguous())
        refuse(PyExc_ValueError, "q must be contiguous [B, Hq, d] with the pool's d and dtype");
    const int B = to_int(q.size(0), "B"), Hq = to_int(q.size(1), "Hq");
    const double scale = a[6] == Py_None ? std::pow((double)p.d, -0.5) : PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) throw Refused{};
    const Table table(pt, B);
    const Scope scope(a[12], q, {&lens, &pt, &kp, &vp, given_o, status, ws, given_lse});
    if (given_o && (given_o->sizes() != q.sizes() || given_o->scalar_type() != q.scalar_type() ||
                    !given_o->is_contiguous()))
        refuse(PyExc_ValueError, "o must be contiguous and of q's shape and dtype");
    if (given_lse &&
        (given_lse->dim() != 2 || given_lse->size(0) != B || given_lse->size(1) != Hq ||
         given_lse->scalar_type() != at::kFloat || !given_lse->is_contiguous()))
        refuse(PyExc_ValueError, "lse must be contiguous float32 [B, Hq]");
    const int32_t* lens_at = int32s(&lens, "seq_lens", B);
    int32_t* status_at = int32s(status, "status", 1);
    const at::Tensor o = given_o ? *given_o : at::empty(q.sizes(), q.options());
    at::Tensor lse;
    if (given_lse) lse = *given_lse;
    else if (a[9] == Py_True) lse = at::empty({B, Hq}, q.options().dtype(at::kFloat));
    const Workspace w(ws, gret_paged_attention_workspace_size(p.dtype, Hq, p.H, p.d));
    check("gret_paged_attention_decode",
          gret_paged_attention_decode(
              q.data_ptr(), lens_at, table.entries, table.stride, table.max_pages, p.k, p.v, p.sp,
              p.st, p.sh, p.n_pages, p.page, p.dtype, (float)scale, window, B, Hq, p.H, p.d,
              o.data_ptr(), lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
              status_at, w.at, w.bytes, scope.raw));
    PyObject* po = given_o ? Py_NewRef(a[8]) : THPVariable_Wrap(o);
    PyObject* pl = a[9] != Py_True ? Py_NewRef(a[9]) : THPVariable_Wrap(lse);
    return Py_BuildValue("(NN)", po, pl);
}

// (k, v, pos, page_table, k_pages, v_pages, cu_seqlens, head_major, status, stream)
PyObject* append(PyObject* const* a) {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &pos = tensor(a[2], "pos"),
                     &pt = tensor(a[3], "page_table"), &kp = tensor(a[4], "k_pages"),
                     &vp = tensor(a[5], "v_pages");
    const at::Tensor *cu = optional(a[6], "cu_seqlens"), *status = optional(a[8], "status");
    const Pool p(kp, vp, to_bool(a[7]));
    if (k.dim() != 3 || k.size(1) != p.H || k.size(2) != p.d || v.sizes() != k.sizes() ||
        k.scalar_type() != kp.scalar_type() || v.scalar_type() != k.scalar_type())
        refuse(PyExc_ValueError, "k and v must be [T, Hkv, d] with the pool's heads and dtype");
    if (k.stride(2) != 1 || v.stride(2) != 1)
        refuse(PyExc_ValueError, "last dimension must be contiguous");
    const int S = to_int(pos.numel(), "rows");
    const Table table(pt, S);
    const Scope scope(a[9], k, {&v, &pos, &pt, &kp, &vp, cu, status});
    check("gret_paged_append",
          gret_paged_append(k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
                            v.stride(1), k.size(0), int32s(cu, "cu_seqlens", (int64_t)S + 1),
                            int32s(&pos, "pos", S), S, table.entries, table.stride,
                            table.max_pages, p.k, p.v, p.sp, p.st, p.sh, p.n_pages, p.page, p.dtype,
                            p.H, p.d, int32s(status, "status", 1), scope.raw));
    Py_RETURN_NONE;
}

// (delta, seq_lens, page_table, ref, k_pages, v_pages, head_major, pos, status, workspace,
// stream)
PyObject* resize(PyObject* const* a) {
    const at::Tensor &delta = tensor(a[0], "delta"), &lens = tensor(a[1], "seq_lens"),
                     &pt = tensor(a[2], "page_table"), &ref = tensor(a[3], "ref"),
                     &kp = tensor(a[4], "k_pages"), &vp = tensor(a[5], "v_pages");
    const at::Tensor *given = optional(a[7], "pos"), *status = optional(a[8], "status"),
                     *ws = optional(a[9], "workspace");
    const int S = to_int(lens.numel(), "rows");
    const Pool p(kp, vp, to_bool(a[6]));
    const Table table(pt, S);
    const Scope scope(a[10], lens, {&delta, &pt, &ref, &kp, &vp, given, status, ws});
    const at::Tensor pos = int32_output(given, S, lens);
    const Workspace w(ws, gret_paged_resize_workspace_size(S));
    check("gret_paged_resize",
          gret_paged_resize(int32s(&delta, "delta", S), int32s(&lens, "seq_lens", S), S,
                            table.entries, table.stride, table.max_pages,
                            int32s(&ref, "ref", p.n_pages), p.k, p.v, p.sp, p.st, p.sh, p.n_pages,
                            p.page, p.dtype, p.H, p.d, int32s(&pos, "pos", S),
                            int32s(status, "status", 1), w.at, w.bytes, scope.raw));
    return given ? Py_NewRef(a[7]) : THPVariable_Wrap(pos);
}

// (src, dst, seq_lens, page_table, ref, page_size, status, stream)
PyObject* fork(PyObject* const* a) {
    const at::Tensor &src = tensor(a[0], "src"), &dst = tensor(a[1], "dst"),
                     &lens = tensor(a[2], "seq_lens"), &pt = tensor(a[3], "page_table"),
                     &ref = tensor(a[4], "ref");
    const int page = to_int(a[5], "page_size");
    const at::Tensor* status = optional(a[6], "status");
    const int S = to_int(lens.numel(), "rows"), n = to_int(src.numel(), "pairs"),
              P = to_int(ref.numel(), "pages");
    const Table table(pt, S);
    const Scope scope(a[7], lens, {&src, &dst, &pt, &ref, status});
    check("gret_paged_fork",
          gret_paged_fork(int32s(&src, "src", n), int32s(&dst, "dst", n), n,
                          int32s(&lens, "seq_lens", S), S, table.entries, table.stride,
                          table.max_pages, int32s(&ref, "ref", P), P, page,
                          int32s(status, "status", 1), scope.raw));
    Py_RETURN_NONE;
}

// (seq_lens, page_table, ref, k_pages, v_pages, head_major, n_live, status, workspace, stream)
PyObject* compact(PyObject* const* a) {
    const at::Tensor &lens = tensor(a[0], "seq_lens"), &pt = tensor(a[1], "page_table"),
                     &ref = tensor(a[2], "ref"), &kp = tensor(a[3], "k_pages"),
                     &vp = tensor(a[4], "v_pages");
    const at::Tensor *given = optional(a[6], "n_live"), *status = optional(a[7], "status"),
                     *ws = optional(a[8], "workspace");
    const int S = to_int(lens.numel(), "rows");
    const Pool p(kp, vp, to_bool(a[5]));
    const Table table(pt, S);
    const Scope scope(a[9], lens, {&pt, &ref, &kp, &vp, given, status, ws});
    const at::Tensor n_live = int32_output(given, 1, lens);
    const Workspace w(ws, gret_paged_compact_workspace_size(p.n_pages));
    check("gret_paged_compact",
          gret_paged_compact(int32s(&lens, "seq_lens", S), S, table.entries, table.stride,
                             table.max_pages, int32s(&ref, "ref", p.n_pages), p.k, p.v, p.sp, p.st,
                             p.sh, p.n_pages, p.page, p.dtype, p.H, p.d,
                             int32s(&n_live, "n_live", 1), int32s(status, "status", 1), w.at,
                             w.bytes, scope.raw));
    return given ? Py_NewRef(a[6]) : THPVariable_Wrap(n_live);
}

PyObject* set_check(PyObject* const* a) {
    Py_XSETREF(check_status, Py_NewRef(a[0]));
    Py_RETURN_NONE;
}

// What Python calls: the number of arguments checked, C++ exceptions turned into Python's.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        if (n != N) refuse(PyExc_TypeError, "%d arguments are needed", N);
        return F(args);
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<attention_decode, 13>("attention_decode"),
                         method<append, 10>("append"),
                         method<resize, 11>("resize"),
                         method<fork, 8>("fork"),
                         method<compact, 10>("compact"),
                         method<set_check, 1>("set_check"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
