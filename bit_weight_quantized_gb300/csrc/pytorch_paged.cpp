// pytorch_paged.cpp -- a CPython extension with the Python binding's hot path of
// the paged cache calls (qmm_kv_append, qmm_paged_attn, qmm_kv4_append, qmm_kv4_read,
// qmm_kv4_attn): it reads the torch
// tensors' types, shapes, strides and addresses directly, allocates the outputs and
// the scratch, and calls the library through a function address.  In Python the
// same checks are some eighty attribute reads, 10 to 15 us of a call that takes the
// GPU 3.  Arguments that do not match return -1: the binding then makes its own
// checks, one by one, for the message.  Built by build.py next to libqmm.so; where
// it is missing the binding calls the same library functions through ctypes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <exception>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qmm.h"

namespace {

using at::Tensor;

// args[i] as a tensor; nullptr for None or anything else (ok says which).
const Tensor *tensor(PyObject *o, bool &ok)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o)) {
        ok = false;
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

bool is_int32(const Tensor &t, int64_t dims)
{
    return t.is_cuda() && t.scalar_type() == at::kInt && t.dim() == dims && t.is_contiguous();
}

// [tokens][heads][D] on the device, the heads of a token back to back
bool is_rows(const Tensor &t, at::ScalarType dt, int64_t tokens, int64_t D)
{
    return t.is_cuda() && t.scalar_type() == dt && t.dim() == 3 && t.size(0) == tokens && t.size(2) == D &&
           t.stride(2) == 1 && (t.size(1) == 1 || t.stride(1) == D);
}

// An uninitialized tensor on the current device, straight from torch's allocator: at::empty
// takes its dispatcher twice, 0.4 us.
Tensor empty(at::IntArrayRef size, at::ScalarType type)
{
    return Tensor(at::detail::empty_generic(size, c10::cuda::CUDACachingAllocator::get(),
                                            c10::DispatchKeySet(c10::DispatchKey::CUDA), type, {}));
}

constexpr int64_t kIntMax = 0x7fffffff;

// The cache and the batch; false if they do not match.
bool fill(qmm_paged_kv &kv, const Tensor &k, const Tensor &v, const Tensor &table, const Tensor &cu, const Tensor &len,
          int64_t tokens)
{
    const at::ScalarType dt = k.scalar_type();
    if (!k.is_cuda() || !v.is_cuda() || (dt != at::kHalf && dt != at::kBFloat16) || v.scalar_type() != dt || k.dim() != 4 ||
        v.sizes() != k.sizes() || v.strides() != k.strides() || k.stride(3) != 1 || !is_int32(table, 2) ||
        !is_int32(cu, 1) || !is_int32(len, 1) || table.size(0) != len.size(0) || cu.size(0) != len.size(0) + 1)
        return false;
    for (int64_t d = 0; d < 4; ++d)
        if (k.size(d) > kIntMax)
            return false;
    if (table.size(0) > kIntMax || table.size(1) > kIntMax || tokens > kIntMax)
        return false;
    kv.k = k.data_ptr();
    kv.v = v.data_ptr();
    kv.page_stride = k.stride(0);
    kv.slot_stride = k.stride(1);
    kv.head_stride = k.stride(2);
    kv.block_table = static_cast<const int32_t *>(table.data_ptr());
    kv.cu_q = static_cast<const int32_t *>(cu.data_ptr());
    kv.kv_len = static_cast<const int32_t *>(len.data_ptr());
    kv.num_pages = static_cast<int>(k.size(0));
    kv.page_size = static_cast<int>(k.size(1));
    kv.blocks = static_cast<int>(table.size(1));
    kv.batch = static_cast<int>(len.size(0));
    kv.tokens = static_cast<int>(tokens);
    kv.kv_heads = static_cast<int>(k.size(2));
    kv.head_dim = static_cast<int>(k.size(3));
    kv.dtype = dt == at::kBFloat16 ? QMM_BF16 : QMM_F16;
    return true;
}

bool as_int(PyObject *o, int &v)
{
    const long t = PyLong_AsLong(o);
    if ((t == -1 && PyErr_Occurred()) || t < INT32_MIN || t > INT32_MAX) {
        PyErr_Clear();
        return false;
    }
    v = static_cast<int>(t);
    return true;
}

// The truth of an argument; -1 where it has none (the binding's own checks say so).
int truth(PyObject *o)
{
    const int t = PyObject_IsTrue(o);
    if (t < 0)
        PyErr_Clear();
    return t;
}

template <typename F>
F address(PyObject *o)
{
    const unsigned long long a = PyLong_AsUnsignedLongLong(o);
    return reinterpret_cast<F>(static_cast<uintptr_t>(a));
}

PyObject *mismatch() { return PyLong_FromLong(-1); }

// The exception being handled as torch raises it in Python: torch.OutOfMemoryError from the
// allocator, for one.
PyObject *raise_current()
{
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
}

using append_fn = decltype(&qmm_kv_append);
using attn_fn = decltype(&qmm_paged_attn);
using scratch_fn = decltype(&qmm_paged_attn_workspace);

// kv_append(fn, k, v, k_cache, v_cache, block_table, cu_q, kv_len, q, q_out,
//           cos_sin, interleaved) -> q_out or None; a status (> 0); -1: mismatch
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 12) {
        PyErr_SetString(PyExc_TypeError, "kv_append takes 12 arguments");
        return nullptr;
    }
    try {
        bool ok = true;
        const Tensor *k = tensor(a[1], ok), *v = tensor(a[2], ok), *kc = tensor(a[3], ok), *vc = tensor(a[4], ok),
                     *table = tensor(a[5], ok), *cu = tensor(a[6], ok), *len = tensor(a[7], ok), *q = tensor(a[8], ok),
                     *q_out = tensor(a[9], ok), *cs = tensor(a[10], ok);
        const int inter = truth(a[11]);
        if (!ok || !k || !v || !kc || !vc || !table || !cu || !len || inter < 0 || k->dim() != 3)
            return mismatch();
        qmm_paged_kv kv;
        const int64_t T = k->size(0), D = k->size(2);
        if (!fill(kv, *kc, *vc, *table, *cu, *len, T) || kv.head_dim != D || k->size(1) != kv.kv_heads)
            return mismatch();
        const at::ScalarType dt = kc->scalar_type();
        if (!is_rows(*k, dt, T, D) || !is_rows(*v, dt, T, D) || v->size(1) != kv.kv_heads || (!q && q_out))
            return mismatch();
        const c10::cuda::CUDAGuard guard(k->device());
        int64_t heads = 0;
        Tensor made;
        if (q) {
            heads = q->size(1);
            if (!is_rows(*q, dt, T, D) || heads > kIntMax)
                return mismatch();
            if (!q_out)
                made = empty({T, heads, D}, dt);
            else if (!q_out->is_contiguous() || !is_rows(*q_out, dt, T, D) || q_out->size(1) != heads)
                return mismatch();
        }
        int64_t rot = 0, rope_len = 0;
        if (cs) {
            if (!cs->is_cuda() || cs->scalar_type() != at::kFloat || cs->dim() != 2 || !cs->is_contiguous() ||
                cs->size(0) > kIntMax || cs->size(1) > kIntMax)
                return mismatch();
            rope_len = cs->size(0);
            rot = cs->size(1);
        }
        const auto stream = c10::cuda::getCurrentCUDAStream(k->get_device()).stream();
        const qmm_status st = address<append_fn>(a[0])(
            &kv, k->data_ptr(), k->stride(0), v->data_ptr(), v->stride(0), q ? q->data_ptr() : nullptr,
            q ? q->stride(0) : 0, !q ? nullptr : q_out ? q_out->data_ptr() : made.data_ptr(), static_cast<int>(heads),
            cs ? static_cast<const float *>(cs->data_ptr()) : nullptr, static_cast<int>(rot),
            static_cast<int>(rope_len), inter, stream);
        if (st != QMM_OK)
            return PyLong_FromLong(st);
        if (made.defined())
            return THPVariable_Wrap(std::move(made));
        Py_INCREF(a[9]);
        return a[9];   // q_out or None
    } catch (...) {
        return raise_current();
    }
}

// paged_attn(fn, scratch_fn, q, k_cache, v_cache, block_table, cu_q, kv_len, max_q,
//            max_kv, scale, causal, window, return_lse, out, workspace)
//   -> out or (out, lse); a status (> 0); -1: mismatch
PyObject *paged_attn(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 16) {
        PyErr_SetString(PyExc_TypeError, "paged_attn takes 16 arguments");
        return nullptr;
    }
    try {
        bool ok = true;
        const Tensor *q = tensor(a[2], ok), *kc = tensor(a[3], ok), *vc = tensor(a[4], ok), *table = tensor(a[5], ok),
                     *cu = tensor(a[6], ok), *len = tensor(a[7], ok), *out = tensor(a[14], ok), *ws = tensor(a[15], ok);
        int max_q, max_kv, window;
        const int causal = truth(a[11]), want_lse = truth(a[13]);
        if (!ok || !q || !kc || !vc || !table || !cu || !len || causal < 0 || want_lse < 0 || q->dim() != 3 ||
            !as_int(a[8], max_q) || !as_int(a[9], max_kv) || !as_int(a[12], window))
            return mismatch();
        qmm_paged_kv kv;
        const int64_t T = q->size(0), heads = q->size(1), D = q->size(2);
        if (!fill(kv, *kc, *vc, *table, *cu, *len, T) || kv.head_dim != D || heads > kIntMax)
            return mismatch();
        const at::ScalarType dt = kc->scalar_type();
        if (!is_rows(*q, dt, T, D))
            return mismatch();
        const double scale = PyFloat_AsDouble(a[10]);
        if (scale == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            return mismatch();
        }
        const c10::cuda::CUDAGuard guard(q->device());
        Tensor made, lse;
        c10::DataPtr scratch;
        if (!out)
            made = empty({T, heads, D}, dt);
        else if (!out->is_contiguous() || !is_rows(*out, dt, T, D) || out->size(1) != heads)
            return mismatch();
        if (want_lse)
            lse = empty({T, heads}, at::kFloat);
        size_t bytes;
        if (ws) {
            if (!ws->is_cuda() || ws->scalar_type() != at::kByte || !ws->is_contiguous())
                return mismatch();
            bytes = static_cast<size_t>(ws->numel());
        } else {
            bytes = address<scratch_fn>(a[1])(static_cast<int>(heads), kv.kv_heads, static_cast<int>(D), max_q);
            scratch = c10::cuda::CUDACachingAllocator::get()->allocate(bytes ? bytes : 16);
        }
        const auto stream = c10::cuda::getCurrentCUDAStream(q->get_device()).stream();
        const qmm_status st = address<attn_fn>(a[0])(
            &kv, q->data_ptr(), q->stride(0), static_cast<int>(heads), static_cast<float>(scale), causal, window,
            out ? out->data_ptr() : made.data_ptr(), want_lse ? static_cast<float *>(lse.data_ptr()) : nullptr, max_q,
            max_kv, ws ? ws->data_ptr() : scratch.get(), bytes, stream);
        if (st != QMM_OK)
            return PyLong_FromLong(st);
        PyObject *o;
        if (out) {
            Py_INCREF(a[14]);
            o = a[14];
        } else if (!(o = THPVariable_Wrap(std::move(made)))) {
            return nullptr;
        }
        if (!want_lse)
            return o;
        PyObject *l = THPVariable_Wrap(std::move(lse));
        PyObject *pair = l ? PyTuple_Pack(2, o, l) : nullptr;
        Py_DECREF(o);
        Py_XDECREF(l);
        return pair;
    } catch (...) {
        return raise_current();
    }
}

// ---- the cache in 4 bits --------------------------------------------------------------
// The cache and the batch from args[0 .. 5] (k_cache, v_cache, scales, block_table, cu_q,
// kv_len); false if they do not match.
bool fill4(qmm_paged_kv4 &kv, PyObject *const *a, int64_t tokens, c10::DeviceIndex &dev)
{
    bool ok = true;
    const Tensor *k = tensor(a[0], ok), *v = tensor(a[1], ok), *sc = tensor(a[2], ok), *table = tensor(a[3], ok),
                 *cu = tensor(a[4], ok), *len = tensor(a[5], ok);
    if (!ok || !k || !v || !sc || !table || !cu || !len || !k->is_cuda() || !v->is_cuda() || !sc->is_cuda())
        return false;
    const at::ScalarType dt = sc->scalar_type();
    if (k->scalar_type() != at::kByte || v->scalar_type() != at::kByte || (dt != at::kHalf && dt != at::kBFloat16) ||
        k->dim() != 4 || sc->dim() != 4 || v->sizes() != k->sizes() || v->strides() != k->strides() ||
        k->stride(3) != 1 || sc->stride(3) != 1 || (k->size(3) != 32 && k->size(3) != 64) ||
        sc->size(3) * 16 != k->size(3) || !is_int32(*table, 2) || !is_int32(*cu, 1) || !is_int32(*len, 1) ||
        table->size(0) != len->size(0) || cu->size(0) != len->size(0) + 1)
        return false;
    dev = k->get_device();
    for (const Tensor *t : {v, sc, table, cu, len})
        if (t->get_device() != dev)
            return false;
    for (int64_t d = 0; d < 3; ++d)
        if (k->size(d) != sc->size(d) || k->size(d) > kIntMax)
            return false;
    if (table->size(0) > kIntMax || table->size(1) > kIntMax || tokens > kIntMax)
        return false;
    kv.k = k->data_ptr();
    kv.v = v->data_ptr();
    kv.page_stride = k->stride(0);
    kv.slot_stride = k->stride(1);
    kv.head_stride = k->stride(2);
    kv.block_table = static_cast<const int32_t *>(table->data_ptr());
    kv.cu_q = static_cast<const int32_t *>(cu->data_ptr());
    kv.kv_len = static_cast<const int32_t *>(len->data_ptr());
    kv.num_pages = static_cast<int>(k->size(0));
    kv.page_size = static_cast<int>(k->size(1));
    kv.blocks = static_cast<int>(table->size(1));
    kv.batch = static_cast<int>(len->size(0));
    kv.tokens = static_cast<int>(tokens);
    kv.kv_heads = static_cast<int>(k->size(2));
    kv.head_dim = static_cast<int>(2 * k->size(3));
    kv.dtype = dt == at::kBFloat16 ? QMM_BF16 : QMM_F16;
    kv.scales = sc->data_ptr();
    kv.scale_page_stride = sc->stride(0);
    kv.scale_slot_stride = sc->stride(1);
    kv.scale_head_stride = sc->stride(2);
    return true;
}

// An optional [n] vector of type dt on the device.
bool is_weight(const Tensor *t, at::ScalarType dt, int64_t n, c10::DeviceIndex dev)
{
    return !t || (t->is_cuda() && t->get_device() == dev && t->scalar_type() == dt && t->dim() == 1 && t->size(0) == n &&
                  t->is_contiguous());
}

using append4_fn = decltype(&qmm_kv4_append);
using read4_fn = decltype(&qmm_kv4_read);
using attn4_fn = decltype(&qmm_kv4_attn);
using more_fn = decltype(&qmm_kv4_attn_more_workspace);

// kv4_append(fn, k, v, k_cache, v_cache, scales, block_table, cu_q, kv_len, q, q_out, cos_sin,
//            interleaved, q_norm, k_norm, eps) -> q_out or None; a status (> 0); -1: mismatch
PyObject *kv4_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 16) {
        PyErr_SetString(PyExc_TypeError, "kv4_append takes 16 arguments");
        return nullptr;
    }
    try {
        bool ok = true;
        const Tensor *k = tensor(a[1], ok), *v = tensor(a[2], ok), *q = tensor(a[9], ok), *q_out = tensor(a[10], ok),
                     *cs = tensor(a[11], ok), *qn = tensor(a[13], ok), *kn = tensor(a[14], ok);
        const int inter = truth(a[12]);
        if (!ok || !k || !v || inter < 0 || k->dim() != 3)
            return mismatch();
        qmm_paged_kv4 kv;
        c10::DeviceIndex dev;
        const int64_t T = k->size(0), D = k->size(2);
        if (!fill4(kv, a + 3, T, dev) || kv.head_dim != D || k->size(1) != kv.kv_heads)
            return mismatch();
        const at::ScalarType dt = kv.dtype == QMM_BF16 ? at::kBFloat16 : at::kHalf;
        if (!is_rows(*k, dt, T, D) || !is_rows(*v, dt, T, D) || v->size(1) != kv.kv_heads || (!q && (q_out || qn)) ||
            k->get_device() != dev || v->get_device() != dev || !is_weight(qn, dt, D, dev) || !is_weight(kn, dt, D, dev))
            return mismatch();
        const double eps = PyFloat_AsDouble(a[15]);
        if (eps == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            return mismatch();
        }
        const c10::cuda::CUDAGuard guard(k->device());
        int64_t heads = 0;
        Tensor made;
        if (q) {
            heads = q->size(1);
            if (!is_rows(*q, dt, T, D) || heads > kIntMax || q->get_device() != dev)
                return mismatch();
            if (!q_out)
                made = empty({T, heads, D}, dt);
            else if (!q_out->is_contiguous() || !is_rows(*q_out, dt, T, D) || q_out->size(1) != heads ||
                     q_out->get_device() != dev)
                return mismatch();
        }
        int64_t rot = 0, rope_len = 0;
        if (cs) {
            if (!cs->is_cuda() || cs->scalar_type() != at::kFloat || cs->dim() != 2 || !cs->is_contiguous() ||
                cs->size(0) > kIntMax || cs->size(1) > kIntMax || cs->get_device() != dev)
                return mismatch();
            rope_len = cs->size(0);
            rot = cs->size(1);
        }
        const auto stream = c10::cuda::getCurrentCUDAStream(dev).stream();
        const qmm_status st = address<append4_fn>(a[0])(
            &kv, k->data_ptr(), k->stride(0), v->data_ptr(), v->stride(0), q ? q->data_ptr() : nullptr,
            q ? q->stride(0) : 0, !q ? nullptr : q_out ? q_out->data_ptr() : made.data_ptr(), static_cast<int>(heads),
            cs ? static_cast<const float *>(cs->data_ptr()) : nullptr, static_cast<int>(rot), static_cast<int>(rope_len),
            inter, qn ? qn->data_ptr() : nullptr, kn ? kn->data_ptr() : nullptr, static_cast<float>(eps), stream);
        if (st != QMM_OK)
            return PyLong_FromLong(st);
        if (made.defined())
            return THPVariable_Wrap(std::move(made));
        Py_INCREF(a[10]);
        return a[10];   // q_out or None
    } catch (...) {
        return raise_current();
    }
}

// A pair of results; takes neither reference.
PyObject *pair_of(PyObject *x, PyObject *y) { return x && y ? PyTuple_Pack(2, x, y) : nullptr; }

// kv4_read(fn, k_cache, v_cache, scales, block_table, cu_q, kv_len, tokens, k_out, v_out)
//   -> (k_out, v_out); a status (> 0); -1: mismatch
PyObject *kv4_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 10) {
        PyErr_SetString(PyExc_TypeError, "kv4_read takes 10 arguments");
        return nullptr;
    }
    try {
        bool ok = true;
        const Tensor *out[2] = {tensor(a[8], ok), tensor(a[9], ok)};
        int tokens;
        if (!ok || !as_int(a[7], tokens) || tokens < 0)
            return mismatch();
        qmm_paged_kv4 kv;
        c10::DeviceIndex dev;
        if (!fill4(kv, a + 1, tokens, dev))
            return mismatch();
        const at::ScalarType dt = kv.dtype == QMM_BF16 ? at::kBFloat16 : at::kHalf;
        const c10::cuda::CUDAGuard guard(c10::Device(c10::DeviceType::CUDA, dev));
        Tensor made[2];
        void *dst[2];
        for (int i = 0; i < 2; ++i) {
            if (!out[i])
                made[i] = empty({tokens, kv.kv_heads, kv.head_dim}, dt);
            else if (!out[i]->is_contiguous() || !is_rows(*out[i], dt, tokens, kv.head_dim) ||
                     out[i]->size(1) != kv.kv_heads || out[i]->get_device() != dev)
                return mismatch();
            dst[i] = out[i] ? out[i]->data_ptr() : made[i].data_ptr();
        }
        const auto stream = c10::cuda::getCurrentCUDAStream(dev).stream();
        const qmm_status st = address<read4_fn>(a[0])(&kv, dst[0], dst[1], stream);
        if (st != QMM_OK)
            return PyLong_FromLong(st);
        PyObject *r[2];
        for (int i = 0; i < 2; ++i) {
            r[i] = out[i] ? a[8 + i] : THPVariable_Wrap(std::move(made[i]));
            if (out[i])
                Py_INCREF(r[i]);
        }
        PyObject *pair = pair_of(r[0], r[1]);
        Py_XDECREF(r[0]);
        Py_XDECREF(r[1]);
        return pair;
    } catch (...) {
        return raise_current();
    }
}

// kv4_attn(fn, scratch_fn, more_fn, q, k_cache, v_cache, scales, block_table, cu_q, kv_len, max_q,
//          max_kv, scale, causal, window, sinks, return_lse, out, workspace)
//   -> out or (out, lse); a status (> 0); -1: mismatch
PyObject *kv4_attn(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 19) {
        PyErr_SetString(PyExc_TypeError, "kv4_attn takes 19 arguments");
        return nullptr;
    }
    try {
        bool ok = true;
        const Tensor *q = tensor(a[3], ok), *out = tensor(a[17], ok), *ws = tensor(a[18], ok);
        int max_q, max_kv, window, sinks;
        const int causal = truth(a[13]), want_lse = truth(a[16]);
        if (!ok || !q || causal < 0 || want_lse < 0 || q->dim() != 3 || !as_int(a[10], max_q) || !as_int(a[11], max_kv) ||
            !as_int(a[14], window) || !as_int(a[15], sinks))
            return mismatch();
        qmm_paged_kv4 kv;
        c10::DeviceIndex dev;
        const int64_t T = q->size(0), heads = q->size(1), D = q->size(2);
        if (!fill4(kv, a + 4, T, dev) || kv.head_dim != D || heads > kIntMax)
            return mismatch();
        const at::ScalarType dt = kv.dtype == QMM_BF16 ? at::kBFloat16 : at::kHalf;
        if (!is_rows(*q, dt, T, D) || q->get_device() != dev)
            return mismatch();
        const double scale = PyFloat_AsDouble(a[12]);
        if (scale == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            return mismatch();
        }
        const c10::cuda::CUDAGuard guard(q->device());
        Tensor made, lse;
        c10::DataPtr scratch;
        if (!out)
            made = empty({T, heads, D}, dt);
        else if (!out->is_contiguous() || !is_rows(*out, dt, T, D) || out->size(1) != heads || out->get_device() != dev)
            return mismatch();
        if (want_lse)
            lse = empty({T, heads}, at::kFloat);
        size_t bytes;
        if (ws) {
            if (!ws->is_cuda() || ws->scalar_type() != at::kByte || !ws->is_contiguous() || ws->get_device() != dev)
                return mismatch();
            bytes = static_cast<size_t>(ws->numel());
        } else {
            bytes = address<scratch_fn>(a[1])(static_cast<int>(heads), kv.kv_heads, static_cast<int>(D), max_q);
            const size_t more = address<more_fn>(a[2])(kv.batch, kv.tokens, static_cast<int>(heads), kv.kv_heads,
                                                       static_cast<int>(D), max_q, max_kv, sinks);
            auto *allocator = c10::cuda::CUDACachingAllocator::get();
            try {
                scratch = allocator->allocate(bytes + more ? bytes + more : 16);
                bytes += more;
            } catch (const c10::OutOfMemoryError &) {
                if (more == 0)
                    throw;
                scratch = allocator->allocate(bytes);   // it does without
            }
        }
        const auto stream = c10::cuda::getCurrentCUDAStream(dev).stream();
        const qmm_status st = address<attn4_fn>(a[0])(
            &kv, q->data_ptr(), q->stride(0), static_cast<int>(heads), static_cast<float>(scale), causal, window, sinks,
            out ? out->data_ptr() : made.data_ptr(), want_lse ? static_cast<float *>(lse.data_ptr()) : nullptr, max_q,
            max_kv, ws ? ws->data_ptr() : scratch.get(), bytes, stream);
        if (st != QMM_OK)
            return PyLong_FromLong(st);
        PyObject *o = out ? a[17] : THPVariable_Wrap(std::move(made));
        if (out)
            Py_INCREF(o);
        if (!want_lse || !o)
            return o;
        PyObject *l = THPVariable_Wrap(std::move(lse));
        PyObject *pair = pair_of(o, l);
        Py_DECREF(o);
        Py_XDECREF(l);
        return pair;
    } catch (...) {
        return raise_current();
    }
}

PyMethodDef methods[] = {
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(kv_append)), METH_FASTCALL,
     "kv_append(fn, k, v, k_cache, v_cache, block_table, cu_q, kv_len, q, q_out, cos_sin, interleaved)"},
    {"paged_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(paged_attn)), METH_FASTCALL,
     "paged_attn(fn, scratch_fn, q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, max_kv, scale, causal, "
     "window, return_lse, out, workspace)"},
    {"kv4_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(kv4_append)), METH_FASTCALL,
     "kv4_append(fn, k, v, k_cache, v_cache, scales, block_table, cu_q, kv_len, q, q_out, cos_sin, interleaved, "
     "q_norm, k_norm, eps)"},
    {"kv4_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(kv4_read)), METH_FASTCALL,
     "kv4_read(fn, k_cache, v_cache, scales, block_table, cu_q, kv_len, tokens, k_out, v_out)"},
    {"kv4_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(kv4_attn)), METH_FASTCALL,
     "kv4_attn(fn, scratch_fn, more_fn, q, k_cache, v_cache, scales, block_table, cu_q, kv_len, max_q, max_kv, scale, causal, "
     "window, sinks, return_lse, out, workspace)"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmmpaged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmmpaged(void) { return PyModule_Create(&module); }
