// Python entry points of the attention sub-layer and the prompt calls: torch
// tensors in, checked, the C calls of moe.h out.
//
// These operators run for a few microseconds, and of the 10 that an append of 8
// tokens took through ctypes, 7.5 were the reading of eight tensors' shapes and
// strides in Python and the conversion of 22 arguments.  Here the same checks
// cost nanoseconds.  A wrong tensor raises ValueError; what the library refuses
// comes back as its return code.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <string>
#include <utility>

#include "moe.h"

namespace {

// A Python exception is set; unwinds to the entry.
struct Raised {};

[[noreturn]] void value_error(const std::string &what) {
    PyErr_SetString(PyExc_ValueError, what.c_str());
    throw Raised{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) {
        PyErr_SetString(PyExc_TypeError, (std::string(name) + ": a tensor").c_str());
        throw Raised{};
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) value_error(std::string(name) + ": a dense tensor");
    return t;
}

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

int32_t int32(PyObject *o, const char *name) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + ": outside 32 bits");
    return static_cast<int32_t>(v);
}

// The cache's description, by its address.
const gqa_pages *pages_at(PyObject *o) {
    const void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised{};
    if (!p) value_error("no cache");
    return static_cast<const gqa_pages *>(p);
}

// A size as the C calls take it; what is too large for them stays too large.
int32_t size32(int64_t n) { return static_cast<int32_t>(n < INT32_MAX ? n : INT32_MAX); }

int current_device() {
    c10::DeviceIndex dev = 0;
    return c10::cuda::GetDevice(&dev) == cudaSuccess ? dev : 0;
}

void on_device(const at::Tensor &t, const char *name, int dev) {
    if (t.get_device() != dev)
        value_error(std::string(name) + ": on " + t.device().str() + ", the current device is cuda:" + std::to_string(dev));
}

cudaStream_t stream_of(PyObject *o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    void *s = PyLong_AsVoidPtr(o);
    if (!s && PyErr_Occurred()) throw Raised{};
    return static_cast<cudaStream_t>(s);
}

// [T, heads, D] bf16 whose rows are contiguous (rows themselves may be strided);
// elements from one row to the next.  heads < 0: any number.
int64_t heads_of(const at::Tensor &t, const char *name, int64_t T, int64_t heads, int64_t D, int dev) {
    if (t.dim() != 3 || t.scalar_type() != at::kBFloat16 || t.size(0) != T || t.size(2) != D || (heads >= 0 && t.size(1) != heads))
        value_error(std::string(name) + ": [" + std::to_string(T) + ", " + (heads < 0 ? "heads" : std::to_string(heads)) + ", " +
                    std::to_string(D) + "] in bf16");
    if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != D))
        value_error(std::string(name) + ": the heads of a row must be contiguous");
    on_device(t, name, dev);
    return T > 1 ? t.stride(0) : t.size(1) * D;
}

// A contiguous int32 array on the device, its first size n (n < 0: any).
const int32_t *ints_of(const at::Tensor &t, const char *name, int64_t n, int dims, int dev) {
    if (t.scalar_type() != at::kInt || t.dim() != dims || (n >= 0 && t.size(0) != n) || !t.is_contiguous())
        value_error(std::string(name) + ": int32, contiguous, " + std::to_string(dims) + " dimension(s)" +
                    (n < 0 ? "" : ", the first " + std::to_string(n)));
    on_device(t, name, dev);
    return static_cast<const int32_t *>(t.data_ptr());
}

int device_of_cache(const char *what, PyObject *device) {
    const int dev = current_device();
    const int64_t want = integer(device);
    if (dev != want)
        value_error(std::string(what) + ": the cache is on cuda:" + std::to_string(want) + ", the current device is cuda:" +
                    std::to_string(dev));
    return dev;
}

// What the linear calls share: q, scale, bias, rows, K, group, x, y from v[0] on.
struct Linear {
    moe_qweight w;
    int32_t N, K, group;
    int64_t B, x_stride, y_stride;
    const void *x;
    void *y;
    bool fp32;
    int dev;

    explicit Linear(PyObject *const *v) {
        const at::Tensor &q = tensor(v[0], "linear: codes"), &s = tensor(v[1], "linear: scales"), &b = tensor(v[2], "linear: biases");
        N = int32(v[3], "rows");
        K = int32(v[4], "K");
        group = int32(v[5], "group");
        const at::Tensor &xt = tensor(v[6], "linear: x"), &yt = tensor(v[7], "linear: y");
        if (xt.dim() != 2 || xt.size(1) != K || xt.scalar_type() != at::kBFloat16 || xt.stride(1) != 1)
            value_error("linear: x [B, " + std::to_string(K) + "] in bf16, its rows contiguous");
        if (q.numel() * 8 != static_cast<int64_t>(N) * K) value_error("linear: one matrix [N, K], not a stack");
        const int64_t pitch = group > 0 ? (K / group + 7) / 8 * 8 : 0;
        if (q.scalar_type() != at::kInt || !q.is_contiguous()) value_error("linear: codes in int32, contiguous");
        for (const at::Tensor *t : {&s, &b})
            if (t->element_size() != 2 || !t->is_contiguous() || t->numel() != N * pitch)
                value_error("linear: scales and biases [N, " + std::to_string(pitch) + "] in 16 bits, contiguous");
        B = xt.size(0);
        fp32 = yt.scalar_type() == at::kFloat;
        if (yt.dim() != 2 || yt.size(0) != B || yt.size(1) != N || !(fp32 || yt.scalar_type() == at::kBFloat16) ||
            (N > 1 && yt.stride(1) != 1))
            value_error("linear: y [B, " + std::to_string(N) + "] in bf16 or fp32, its rows contiguous");
        dev = current_device();
        on_device(xt, "linear: x", dev);
        on_device(yt, "linear: y", dev);
        on_device(q, "linear: codes", dev);
        on_device(s, "linear: scales", dev);
        on_device(b, "linear: biases", dev);
        w = {static_cast<const uint32_t *>(q.data_ptr()), static_cast<const uint16_t *>(s.data_ptr()),
             static_cast<const uint16_t *>(b.data_ptr())};
        x = xt.data_ptr();
        y = yt.data_ptr();
        x_stride = B > 1 ? xt.stride(0) : K;
        y_stride = B > 1 ? yt.stride(0) : N;
    }
};

// An int32 tensor for errors found on the device, or None.
int32_t *status_of(PyObject *o, const char *name, int dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    on_device(t, name, dev);
    if (t.scalar_type() != at::kInt || t.numel() < 1) value_error(std::string(name) + " in int32");
    return static_cast<int32_t *>(t.data_ptr());
}

// A call's scratch and its bytes.
std::pair<void *, size_t> scratch_of(PyObject *o, int dev) {
    const at::Tensor &ws = tensor(o, "ws");
    if (ws.get_device() != dev || !ws.is_contiguous()) value_error("ws: contiguous, on the current device");
    return {ws.data_ptr(), static_cast<size_t>(ws.numel()) * ws.element_size()};
}

// q, scale, bias, rows, K, group, x, y, status | None, stream | None
int linear(PyObject *const *v) {
    const Linear l(v);
    return int4_linear(&l.w, l.N, l.K, l.group, l.x, l.x_stride, size32(l.B), l.y, l.y_stride, l.fp32,
                       status_of(v[8], "linear: status", l.dev), stream_of(v[9], l.dev));
}

// q, scale, bias, rows, K, group, x, y, ws, status | None, stream | None
int linear_prompt(PyObject *const *v) {
    const Linear l(v);
    const auto [ws, bytes] = scratch_of(v[8], l.dev);
    return int4_linear_prompt(&l.w, l.N, l.K, l.group, l.x, l.x_stride, size32(l.B), l.y, l.y_stride, l.fp32, ws, bytes,
                              status_of(v[9], "linear: status", l.dev), stream_of(v[10], l.dev));
}

// pages, device, status (addresses and a number), q | None, k, v, seq, index, page_table, inv_freq | None,
// pos_offset, interleaved, q_out | None, stream | None
int append(PyObject *const *v) {
    const int dev = device_of_cache("append", v[1]);
    const gqa_pages *pages = pages_at(v[0]);
    auto *status = static_cast<int32_t *>(PyLong_AsVoidPtr(v[2]));
    if (!status && PyErr_Occurred()) throw Raised{};
    const at::Tensor &k = tensor(v[4], "k"), &val = tensor(v[5], "v");
    const int64_t T = k.dim() ? k.size(0) : 0;
    const int64_t ks = heads_of(k, "k", T, pages->Hkv, pages->D, dev), vs = heads_of(val, "v", T, pages->Hkv, pages->D, dev);
    const int32_t *seq = ints_of(tensor(v[6], "seq"), "seq", T, 1, dev);
    const int32_t *index = ints_of(tensor(v[7], "index"), "index", T, 1, dev);
    const at::Tensor &table = tensor(v[8], "page_table");
    const int32_t *at = ints_of(table, "page_table", -1, 2, dev);
    const float *freq = nullptr;
    int64_t rot = 0;
    if (v[9] != Py_None) {
        const at::Tensor &f = tensor(v[9], "inv_freq");
        if (f.scalar_type() != at::kFloat || f.dim() != 1 || !f.is_contiguous() || f.get_device() != dev)
            value_error("inv_freq: fp32 [rot / 2], contiguous, on the current device");
        rot = 2 * f.size(0);
        freq = static_cast<const float *>(f.data_ptr());
    }
    int64_t Hq = 0, qs = 0, os = 0;
    const void *q_at = nullptr;
    void *out_at = nullptr;
    if (v[3] == Py_None) {
        if (v[12] != Py_None) value_error("q_out without q");
    } else {
        const at::Tensor &q = tensor(v[3], "q"), &out = tensor(v[12], "q_out");
        qs = heads_of(q, "q", T, -1, pages->D, dev);
        Hq = q.size(1);
        os = heads_of(out, "q_out", T, Hq, pages->D, dev);
        q_at = q.data_ptr();
        out_at = out.data_ptr();
    }
    const int32_t offset = int32(v[10], "pos_offset");
    const int turned = PyObject_IsTrue(v[11]);
    if (turned < 0) throw Raised{};
    return gqa_append(pages, q_at, qs, k.data_ptr(), ks, val.data_ptr(), vs, size32(T), size32(Hq), seq, index, at,
                      size32(table.size(0)), size32(table.size(1)), offset, freq, size32(rot), turned, out_at, os, status,
                      stream_of(v[13], dev));
}

// The pages of prefix_len shared positions (NULL if there are none).
const int32_t *prefix_of(PyObject *o, int32_t prefix_len, const gqa_pages *pages, int dev) {
    if (!prefix_len) return nullptr;
    if (o == Py_None) value_error("prefix_len without prefix_pages");
    const at::Tensor &t = tensor(o, "prefix_pages");
    const int32_t *at = ints_of(t, "prefix_pages", -1, 1, dev);
    if (prefix_len > t.size(0) * pages->page_size) value_error("prefix_pages: too few for prefix_len");
    return at;
}

// pages, device, q, page_table, seq_len, prefix_pages | None, prefix_len, scale, out, ws, stream | None and,
// where the workspace is this call's own (its control block is then cleared first), the address for errors
int attend(PyObject *const *v) {
    const int dev = device_of_cache("attend", v[1]);
    const gqa_pages *pages = pages_at(v[0]);
    const at::Tensor &q = tensor(v[2], "q");
    const int64_t B = q.dim() ? q.size(0) : 0, qs = heads_of(q, "q", B, -1, pages->D, dev);
    const at::Tensor &table = tensor(v[3], "page_table");
    const int32_t *at = ints_of(table, "page_table", B, 2, dev);
    const int32_t *lens = ints_of(tensor(v[4], "seq_len"), "seq_len", B, 1, dev);
    const int32_t prefix_len = int32(v[6], "prefix_len");
    const int32_t *prefix = prefix_of(v[5], prefix_len, pages, dev);
    const double scale = PyFloat_AsDouble(v[7]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const at::Tensor &out = tensor(v[8], "out");
    const int64_t os = heads_of(out, "out", B, q.size(1), pages->D, dev);
    const auto [ws, bytes] = scratch_of(v[9], dev);
    const cudaStream_t stream = stream_of(v[10], dev);
    auto *status = static_cast<int32_t *>(ws);
    if (v[11] != Py_None) {
        status = static_cast<int32_t *>(PyLong_AsVoidPtr(v[11]));
        if (!status && PyErr_Occurred()) throw Raised{};
        const int rc = moe_workspace_init(ws, bytes, stream);
        if (rc) return rc;
    }
    return gqa_paged_attention_status(pages, q.data_ptr(), qs, size32(B), size32(q.size(1)), prefix, prefix_len, at,
                                      size32(table.size(1)), lens, static_cast<float>(scale), out.data_ptr(), os,
                                      ws, bytes, status, stream);
}

// pages, device, q, q_start, page_table, seq_len, prefix_pages | None, prefix_len, scale, out, ws, stream | None,
// and the address for errors where it is not the workspace
int attend_prompt(PyObject *const *v) {
    const int dev = device_of_cache("attend_prompt", v[1]);
    const gqa_pages *pages = pages_at(v[0]);
    const at::Tensor &q = tensor(v[2], "q");
    const int64_t T = q.dim() ? q.size(0) : 0, qs = heads_of(q, "q", T, -1, pages->D, dev);
    const at::Tensor &lens = tensor(v[5], "seq_len");
    const int32_t *len = ints_of(lens, "seq_len", -1, 1, dev);
    const int64_t n_seq = lens.size(0);
    const int32_t *start = ints_of(tensor(v[3], "q_start"), "q_start", n_seq + 1, 1, dev);
    const at::Tensor &table = tensor(v[4], "page_table");
    const int32_t *at = ints_of(table, "page_table", n_seq, 2, dev);
    const int32_t prefix_len = int32(v[7], "prefix_len");
    const int32_t *prefix = prefix_of(v[6], prefix_len, pages, dev);
    const double scale = PyFloat_AsDouble(v[8]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const at::Tensor &out = tensor(v[9], "out");
    const int64_t os = heads_of(out, "out", T, q.size(1), pages->D, dev);
    const auto [ws, bytes] = scratch_of(v[10], dev);
    auto *status = static_cast<int32_t *>(ws);
    if (v[12] != Py_None) {
        status = static_cast<int32_t *>(PyLong_AsVoidPtr(v[12]));
        if (!status && PyErr_Occurred()) throw Raised{};
    }
    return gqa_prompt_attention(pages, q.data_ptr(), qs, size32(T), size32(q.size(1)), start, size32(n_seq), prefix,
                                prefix_len, at, size32(table.size(1)), len, static_cast<float>(scale), out.data_ptr(),
                                os, ws, bytes, status, stream_of(v[11], dev));
}

// A contiguous result of token_logprobs, or None: its address.
template <typename E>
E *result_of(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape, int dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || !t.is_contiguous() || t.sizes() != at::IntArrayRef(shape))
        value_error(std::string(name) + ": " + (type == at::kFloat ? "fp32" : "int32") + ", contiguous, a value a row" +
                    (shape.size() > 1 ? " and alternative" : ""));
    on_device(t, name, dev);
    return static_cast<E *>(t.data_ptr());
}

// Rows of scores and the tokens given for them.
struct Scores {
    const at::Tensor &x;
    bool fp32;
    int dev;
    int64_t T, V;
    int32_t n_top;
    const int32_t *targets;

    Scores(PyObject *logits, PyObject *given, PyObject *n) : x(tensor(logits, "logits")), dev(current_device()) {
        fp32 = x.scalar_type() == at::kFloat;
        if (x.dim() != 2 || !(fp32 || x.scalar_type() == at::kBFloat16) || (x.size(1) > 1 && x.stride(1) != 1))
            value_error("logits: [T, V] in fp32 or bf16, its rows contiguous");
        on_device(x, "logits", dev);
        T = x.size(0);
        V = x.size(1);
        n_top = int32(n, "n_top");
        targets = given == Py_None ? nullptr : ints_of(tensor(given, "targets"), "targets", T, 1, dev);
    }
    // ws_: None for scratch of the call's own; fill: the results hold nothing yet
    int call(float *logprob, float *entropy, int32_t *ids, float *top, PyObject *ws_, PyObject *status_, PyObject *stream,
             bool fill) const {
        at::Tensor own;
        std::pair<void *, size_t> scratch{nullptr, 0};
        if (ws_ == Py_None) {
            scratch.second = token_logprobs_workspace_bytes(size32(T), size32(V), n_top);
            own = at::empty({static_cast<int64_t>(scratch.second)}, x.options().dtype(at::kByte));
            scratch.first = own.data_ptr();
        } else {
            scratch = scratch_of(ws_, dev);
        }
        const auto [ws, bytes] = scratch;
        int32_t *status = status_ == Py_None ? static_cast<int32_t *>(ws) : status_of(status_, "status", dev);
        return (fill ? token_logprobs_filled : token_logprobs)(x.data_ptr(), T > 1 ? x.stride(0) : V, fp32, size32(T),
                                                               size32(V), targets, logprob, entropy, n_top, ids, top, ws,
                                                               bytes, status, stream_of(stream, dev));
    }
};

// logits, targets | None, logprob | None, entropy | None, n_top, top_ids | None, top_logprobs | None, ws | None,
// status | None (errors then go to the workspace), stream | None, and whether padding rows' results are filled in
int scores(PyObject *const *v) {
    const Scores s(v[0], v[1], v[4]);
    float *logprob = result_of<float>(v[2], "logprob", at::kFloat, {s.T}, s.dev);
    float *entropy = result_of<float>(v[3], "entropy", at::kFloat, {s.T}, s.dev);
    int32_t *ids = s.n_top > 0 ? result_of<int32_t>(v[5], "top_ids", at::kInt, {s.T, s.n_top}, s.dev) : nullptr;
    float *top = s.n_top > 0 ? result_of<float>(v[6], "top_logprobs", at::kFloat, {s.T, s.n_top}, s.dev) : nullptr;
    return s.call(logprob, entropy, ids, top, v[7], v[8], v[9], v[10] == Py_True);
}

// logits, targets | None, n_top, ws | None, status | None, stream | None: scores with results of its own (made in
// Python they took longer than one row's kernels): (rc, logprob | None, entropy, top_ids, top_logprobs)
PyObject *scores_new(PyObject *const *v) {
    const Scores s(v[0], v[1], v[2]);
    if (s.n_top < 0) value_error("n_top: 0 at least");
    // (more alternatives than there can be are refused before memory for them is asked for)
    if (!token_logprobs_workspace_bytes(size32(s.T), size32(s.V), s.n_top))
        return Py_BuildValue("(iOOOO)", s.T < 1 || s.T > 1 << 24 ? MOE_ERR_TOKENS : MOE_ERR_SHAPE, Py_None, Py_None, Py_None, Py_None);
    const auto f = s.x.options().dtype(at::kFloat);
    const at::Tensor logprob = s.targets ? at::empty({s.T}, f) : at::Tensor(), entropy = at::empty({s.T}, f),
                     ids = at::empty({s.T, s.n_top}, f.dtype(at::kInt)), top = at::empty({s.T, s.n_top}, f);
    const int rc = s.call(s.targets ? static_cast<float *>(logprob.data_ptr()) : nullptr, static_cast<float *>(entropy.data_ptr()),
                          s.n_top ? static_cast<int32_t *>(ids.data_ptr()) : nullptr,
                          s.n_top ? static_cast<float *>(top.data_ptr()) : nullptr, v[3], v[4], v[5], true);
    // (N takes the references; a missing one has set an exception)
    PyObject *given = s.targets ? THPVariable_Wrap(logprob) : Py_NewRef(Py_None);
    return Py_BuildValue("(iNNNN)", rc, given, THPVariable_Wrap(entropy), THPVariable_Wrap(ids), THPVariable_Wrap(top));
}

PyObject *as_object(int rc) { return PyLong_FromLong(rc); }
PyObject *as_object(PyObject *o) { return o; }

// ARGS arguments, and up to MORE that are None if they are left out.
template <auto CALL, int ARGS, int MORE>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n < ARGS || n > ARGS + MORE) {
        PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", ARGS, n);
        return nullptr;
    }
    PyObject *all[ARGS + MORE];
    for (Py_ssize_t i = 0; i < ARGS + MORE; ++i) all[i] = i < n ? args[i] : Py_None;
    try {
        return as_object(CALL(all));
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <auto CALL, int ARGS, int MORE = 0>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<CALL, ARGS, MORE>));
}

PyMethodDef methods[] = {{"linear", fast<linear, 10>(), METH_FASTCALL, "int4_linear"},
                         {"append", fast<append, 14>(), METH_FASTCALL, "gqa_append"},
                         {"attend", fast<attend, 11, 1>(), METH_FASTCALL, "gqa_paged_attention"},
                         {"linear_prompt", fast<linear_prompt, 11>(), METH_FASTCALL, "int4_linear_prompt"},
                         {"attend_prompt", fast<attend_prompt, 12, 1>(), METH_FASTCALL, "gqa_prompt_attention"},
                         {"scores", fast<scores, 10, 1>(), METH_FASTCALL, "token_logprobs"},
                         {"scores_new", fast<scores_new, 6>(), METH_FASTCALL, "token_logprobs"},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "The attention sub-layer's and the prompt's calls on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
