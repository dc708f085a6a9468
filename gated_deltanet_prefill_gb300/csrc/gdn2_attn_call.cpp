// The calls of attn.py once their tensors' metadata are known (CPython module).
//
// A decode step calls the attention-layer operators with a few microseconds of GPU
// work each, where the host sets the time.  attn.py checks the arguments and works
// out the dims struct; this module keeps the struct per set of shapes, strides,
// dtypes and options (nothing is kept by address or content), and makes the call
// for tensors that match one: it allocates the outputs and the workspace and calls
// the library.  A function returns NotImplemented for metadata that it does not
// know; attn.py then checks them and calls again with the dims struct.
// Back to back on the GB300's host (Grace), this module against the same through
// ctypes with the plans cached: qk_norm_rope of one token 5.9 and 17.2 us, append_kv
// of 128 tokens 6.2 and 20.9, paged_attn_fwd of one token 9.8 and 25.5 (there the GPU
// needs 13 by itself when its calls do not overlap).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <unordered_map>

#include "gdn2_attn.h"

namespace {

decltype(&gdn2_qk_norm_rope) qk_norm_rope_fn = nullptr;
decltype(&gdn2_kv_append) kv_append_fn = nullptr;
decltype(&gdn2_paged_attn_workspace_bytes) paged_attn_workspace_fn = nullptr;
decltype(&gdn2_paged_attn_fwd) paged_attn_fn = nullptr;
PyObject *raise_error = nullptr;  // raise_error(status, call)

constexpr size_t kMostPlans = 512;

// Metadata of a call: 64-bit words.
struct Key {
    static constexpr int kWords = 96;
    int64_t w[kWords];
    int n = 0;
    void add(int64_t x) { w[n++] = x; }
    void add(double x) {
        int64_t bits;
        std::memcpy(&bits, &x, 8);
        add(bits);
    }
    // a strided tensor, null: none
    void rows(const at::Tensor *t) {
        if (!t) return add(int64_t{-1});
        const auto size = t->sizes(), stride = t->strides();
        const size_t dim = size.size();
        add(static_cast<int64_t>(dim | static_cast<size_t>(t->scalar_type()) << 8 | static_cast<size_t>(t->is_cuda()) << 16));
        if (dim > 4) return;  // never a known one
        for (size_t i = 0; i < dim; ++i) {
            add(size[i]);
            add(stride[i]);
        }
    }
    // a tensor that has to be contiguous
    void flat(const at::Tensor *t) {
        if (!t) return add(int64_t{-1});
        add(static_cast<int64_t>(static_cast<size_t>(t->scalar_type()) << 8 | static_cast<size_t>(t->is_cuda() && t->is_contiguous()) << 16));
        add(t->numel());
    }
    bool operator==(const Key &o) const { return n == o.n && std::memcmp(w, o.w, n * 8) == 0; }
};
struct Hash {
    size_t operator()(const Key &k) const {
        uint64_t h = 0x9e3779b97f4a7c15ull;
        for (int i = 0; i < k.n; ++i) {
            h = (h ^ static_cast<uint64_t>(k.w[i])) * 0xff51afd7ed558ccdull;
            h ^= h >> 32;
        }
        return static_cast<size_t>(h);
    }
};
struct Plan {
    gdn2_attn_dims dims;
    size_t workspace;
};
using Plans = std::unordered_map<Key, Plan, Hash>;

// The arguments of a call, taken one by one.  `ok` turns false where one is not
// what the call takes.
struct Args {
    PyObject *const *a;
    Py_ssize_t n, i = 0;
    bool ok = true;
    PyObject *next() { return i < n ? a[i++] : Py_None; }
    const at::Tensor *tensor() {
        PyObject *o = next();
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    double number() {
        const double x = PyFloat_AsDouble(next());
        if (x == -1.0 && PyErr_Occurred()) ok = false;
        return x;
    }
    int64_t integer() {
        const long long x = PyLong_AsLongLong(next());
        if (x == -1 && PyErr_Occurred()) ok = false;
        return x;
    }
    bool flag() {
        const int x = PyObject_IsTrue(next());
        if (x < 0) ok = false;
        return x > 0;
    }
};

// Whether a workspace that the caller passed is plain memory on the device of `like`
// (the library gets its address and its bytes); sets an exception if not.
bool workspace_ok(const Args &args, const at::Tensor *workspace, const at::Tensor *like) {
    if (!args.ok || !workspace || (workspace->device() == like->device() && workspace->is_contiguous())) return true;
    PyErr_SetString(PyExc_ValueError, "workspace must be contiguous, on the device of the inputs");
    return false;
}

// Whether a call's tensors are all on one device; sets an exception if not.
bool one_device(const Args &args, std::initializer_list<const at::Tensor *> tensors) {
    const at::Tensor *first = nullptr;
    for (const at::Tensor *t : tensors) {
        if (!args.ok || !t) continue;
        if (!first) first = t;
        if (t->device() == first->device()) continue;
        PyErr_SetString(PyExc_ValueError, "the tensors of a call must be on one device");
        return false;
    }
    return true;
}

// The plan of the call: the known one, or the one that `dims` (bytes of the struct)
// brings.  Returns false where there is none, with or without an exception set.
bool find(Plans &plans, const Key &key, Args &args, Plan &plan) {
    PyObject *dims = args.next();
    if (!args.ok) {
        if (dims == Py_None) PyErr_Clear();
        else if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "a tensor was expected");
        return false;
    }
    const auto it = plans.find(key);
    if (it != plans.end()) {
        plan = it->second;
        return true;
    }
    if (dims == Py_None) return false;
    char *bytes;
    Py_ssize_t size;
    if (PyBytes_AsStringAndSize(dims, &bytes, &size) < 0) return false;
    if (size != static_cast<Py_ssize_t>(sizeof(gdn2_attn_dims))) {
        PyErr_SetString(PyExc_ValueError, "the dims struct has another size");
        return false;
    }
    std::memcpy(&plan.dims, bytes, sizeof(gdn2_attn_dims));
    plan.workspace = paged_attn_workspace_fn(&plan.dims);
    if (plans.size() >= kMostPlans) plans.clear();
    plans.emplace(key, plan);
    return true;
}
PyObject *unknown() {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NOTIMPLEMENTED;
}

void *data(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }
at::Tensor empty(at::IntArrayRef size, at::ScalarType dtype, const at::Tensor &like) {
    return at::Tensor(at::detail::empty_cuda(size, dtype, like.device(), std::nullopt));
}
// Where the call runs: the stream given (an address), or the current one of the
// tensor's device.  The calls make that device the current one first (CUDAGuard): the
// library launches on the current device, whatever its pointers are.
struct Stream {
    void *handle = nullptr;
    bool other = false;  // not the current one
    c10::DeviceIndex device;
    Stream(PyObject *o, const at::Tensor &t) : device(t.device().index()) {
        void *const current = c10::cuda::getCurrentCUDAStream(device).stream();
        handle = o == Py_None ? current : PyLong_AsVoidPtr(o);
        other = handle != current;
    }
    // Memory made here belongs to the current stream: where the call runs on another,
    // it must not be handed out again before that one has passed this point.
    void keep(std::initializer_list<const at::Tensor *> made) const {
        if (!other) return;
        for (const at::Tensor *t : made)
            if (t->defined())
                c10::cuda::CUDACachingAllocator::recordStream(
                    t->storage().data_ptr(), c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), device));
    }
};
PyObject *failed(gdn2_status st, const char *what) {
    PyObject *r = PyObject_CallFunction(raise_error, "is", static_cast<int>(st), what);
    Py_XDECREF(r);
    return nullptr;
}
// A new reference: the tensor as it was passed, or the one made here.
PyObject *result(PyObject *passed, const at::Tensor &made) {
    if (passed == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(passed);
    return passed;
}

// q, k, positions, inv_freq, rope_factor, interleaved, norm, q_weight, k_weight,
// eps, q_out, k_out, stream[, dims] -> (q_out, k_out)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    static Plans plans;
    Args args{a, n};
    Key key;
    const at::Tensor *q = args.tensor(), *k = args.tensor(), *positions = args.tensor(), *inv_freq = args.tensor();
    key.add(args.number());
    key.add(static_cast<int64_t>(args.flag()));
    key.add(static_cast<int64_t>(args.flag()));
    const at::Tensor *q_weight = args.tensor(), *k_weight = args.tensor();
    key.add(args.number());
    const at::Tensor *q_out = args.tensor(), *k_out = args.tensor();
    PyObject *stream = args.next();
    if (!q) args.ok = false;
    if (!one_device(args, {q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out})) return nullptr;
    for (const at::Tensor *t : {q, k, q_out, k_out}) key.rows(t);
    for (const at::Tensor *t : {positions, inv_freq, q_weight, k_weight}) key.flat(t);
    Plan plan;
    if (!find(plans, key, args, plan)) return unknown();
    const gdn2_attn_dims &d = plan.dims;
    const c10::cuda::CUDAGuard guard(q->device());
    const Stream s(stream, *q);
    if (PyErr_Occurred()) return nullptr;
    at::Tensor qo, ko;
    if (!q_out) q_out = &(qo = empty({d.T_tot, d.HQ, d.D}, q->scalar_type(), *q));
    if (!k_out && k) k_out = &(ko = empty({d.T_tot, d.HKV, d.D}, k->scalar_type(), *k));
    void *const p[] = {data(q), data(k), data(q_weight), data(k_weight), data(inv_freq), data(positions), data(q_out), data(k_out)};
    gdn2_status st;
    Py_BEGIN_ALLOW_THREADS
    st = qk_norm_rope_fn(p[0], p[1], p[2], p[3], static_cast<const double *>(p[4]), p[5], p[6], p[7], &d, s.handle);
    Py_END_ALLOW_THREADS
    s.keep({&qo, &ko});
    if (st != GDN2_OK) return failed(st, "gdn2_qk_norm_rope");
    PyObject *r0 = result(a[10], qo), *r1 = k ? result(a[11], ko) : Py_NewRef(Py_None);
    return Py_BuildValue("(NN)", r0, r1);
    END_HANDLE_TH_ERRORS
}

// k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens, q, positions, inv_freq,
// rope_factor, interleaved, norm, q_weight, k_weight, eps, q_out, workspace, stream
// [, dims] -> q_out, or None without q
PyObject *append_kv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    static Plans plans;
    Args args{a, n};
    Key key;
    const at::Tensor *k = args.tensor(), *v = args.tensor(), *k_cache = args.tensor(), *v_cache = args.tensor(),
                     *table = args.tensor(), *lens = args.tensor(), *cu = args.tensor(), *q = args.tensor(),
                     *positions = args.tensor(), *inv_freq = args.tensor();
    key.add(args.number());
    key.add(static_cast<int64_t>(args.flag()));
    key.add(static_cast<int64_t>(args.flag()));
    const at::Tensor *q_weight = args.tensor(), *k_weight = args.tensor();
    key.add(args.number());
    const at::Tensor *q_out = args.tensor(), *workspace = args.tensor();
    PyObject *stream = args.next();
    if (!k || !v || !k_cache || !v_cache || !table || !lens || !cu) args.ok = false;
    if (!workspace_ok(args, workspace, k) ||
        !one_device(args, {k, v, k_cache, v_cache, table, lens, cu, q, positions, inv_freq, q_weight, k_weight, q_out}))
        return nullptr;
    for (const at::Tensor *t : {k, v, k_cache, v_cache, table, q, q_out}) key.rows(t);
    for (const at::Tensor *t : {lens, cu, positions, inv_freq, q_weight, k_weight}) key.flat(t);
    Plan plan;
    if (!find(plans, key, args, plan)) return unknown();
    const gdn2_attn_dims &d = plan.dims;
    const c10::cuda::CUDAGuard guard(k->device());
    const Stream s(stream, *k);
    if (PyErr_Occurred()) return nullptr;
    at::Tensor qo, ws;
    if (!q_out && q) q_out = &(qo = empty({d.T_tot, d.HQ, d.D}, q->scalar_type(), *q));
    if (!workspace) workspace = &(ws = empty({64}, at::kByte, *k));
    void *const p[] = {data(q), data(k), data(v), data(q_weight), data(k_weight), data(inv_freq), data(positions), data(cu),
                       data(lens), data(table), data(q_out), data(k_cache), data(v_cache), data(workspace)};
    const size_t bytes = workspace->nbytes();
    gdn2_status st;
    Py_BEGIN_ALLOW_THREADS
    st = kv_append_fn(p[0], p[1], p[2], p[3], p[4], static_cast<const double *>(p[5]), p[6], p[7],
                      static_cast<const int32_t *>(p[8]), static_cast<const int32_t *>(p[9]), p[10], p[11], p[12], &d, p[13],
                      bytes, s.handle);
    Py_END_ALLOW_THREADS
    s.keep({&qo, &ws});
    if (st != GDN2_OK) return failed(st, "gdn2_kv_append");
    if (!q) Py_RETURN_NONE;
    return result(a[16], qo);
    END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, scale, causal, window_left,
// out, lse, return_lse, workspace, stream[, dims] -> out, or (out, lse)
PyObject *paged_attn_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    static Plans plans;
    Args args{a, n};
    Key key;
    const at::Tensor *q = args.tensor(), *k_cache = args.tensor(), *v_cache = args.tensor(), *table = args.tensor(),
                     *lens = args.tensor(), *cu = args.tensor();
    float scale = 0.f;  // to the library: 1/sqrt(D)
    if (args.a[args.i] == Py_None) {
        ++args.i;
    } else {
        scale = static_cast<float>(args.number());
        if (args.ok && !(scale > 0.f)) {
            PyErr_SetString(PyExc_ValueError, "scale must be positive (None means 1/sqrt(D))");
            return nullptr;
        }
    }
    key.add(static_cast<int64_t>(args.flag()));
    key.add(args.integer());
    const at::Tensor *out = args.tensor(), *lse = args.tensor();
    const bool return_lse = args.flag();
    const at::Tensor *workspace = args.tensor();
    PyObject *stream = args.next();
    if (!q || !k_cache || !v_cache || !table || !lens || !cu) args.ok = false;
    if (!workspace_ok(args, workspace, q) || !one_device(args, {q, k_cache, v_cache, table, lens, cu, out, lse})) return nullptr;
    for (const at::Tensor *t : {q, k_cache, v_cache, table, out}) key.rows(t);
    for (const at::Tensor *t : {lens, cu, lse}) key.flat(t);
    Plan plan;
    if (!find(plans, key, args, plan)) return unknown();
    const gdn2_attn_dims &d = plan.dims;
    const c10::cuda::CUDAGuard guard(q->device());
    const Stream s(stream, *q);
    if (PyErr_Occurred()) return nullptr;
    at::Tensor o, l, ws;
    if (!out) out = &(o = empty({d.T_tot, d.HQ, d.D}, q->scalar_type(), *q));
    if (!lse && return_lse) lse = &(l = empty({d.T_tot, d.HQ}, at::kFloat, *q));
    if (!workspace) workspace = &(ws = empty({static_cast<int64_t>(plan.workspace > 64 ? plan.workspace : 64)}, at::kByte, *q));
    void *const p[] = {data(q), data(k_cache), data(v_cache), data(cu), data(lens), data(table), data(out), data(lse), data(workspace)};
    const size_t bytes = workspace->nbytes();
    gdn2_status st;
    Py_BEGIN_ALLOW_THREADS
    st = paged_attn_fn(p[0], p[1], p[2], p[3], static_cast<const int32_t *>(p[4]), static_cast<const int32_t *>(p[5]),
                       scale, p[6], static_cast<float *>(p[7]), &d, p[8], bytes, s.handle);
    Py_END_ALLOW_THREADS
    s.keep({&o, &l, &ws});
    if (st != GDN2_OK) return failed(st, "gdn2_paged_attn_fwd");
    PyObject *r = result(a[9], o);
    if (!return_lse) return r;
    return Py_BuildValue("(NN)", r, result(a[10], l));
    END_HANDLE_TH_ERRORS
}

// Addresses of the library's four functions, and what raises a status.
PyObject *bind(PyObject *, PyObject *args) {
    unsigned long long f[4];
    PyObject *raise;
    if (!PyArg_ParseTuple(args, "KKKKO", &f[0], &f[1], &f[2], &f[3], &raise)) return nullptr;
    qk_norm_rope_fn = reinterpret_cast<decltype(qk_norm_rope_fn)>(f[0]);
    kv_append_fn = reinterpret_cast<decltype(kv_append_fn)>(f[1]);
    paged_attn_workspace_fn = reinterpret_cast<decltype(paged_attn_workspace_fn)>(f[2]);
    paged_attn_fn = reinterpret_cast<decltype(paged_attn_fn)>(f[3]);
    Py_INCREF(raise);
    Py_XDECREF(raise_error);
    raise_error = raise;
    Py_RETURN_NONE;
}

#define FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"qk_norm_rope", FASTCALL(qk_norm_rope), nullptr},
                         {"append_kv", FASTCALL(append_kv), nullptr},
                         {"paged_attn_fwd", FASTCALL(paged_attn_fwd), nullptr},
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdn2_attn_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gdn2_attn_call() { return PyModule_Create(&module); }
