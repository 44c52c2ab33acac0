// kda_tree_py.cpp -- Python marshalling of the draft-tree, linear-attention and rotary entry points.
//
// A speculative round makes one call of these per layer and operator, on tensors of a few rows.  Marshalled through
// ctypes, a call cost more time on the host than its kernel takes on the GPU: 11.5 us for a step, 9 for a commit,
// 7.5 for a convolution, 10 for a verification, of which a launch is 3.  The same checks on the tensors' own fields, and
// that they share a device, leave 4.0, 3.3, 2.7 and 3.3 us.  The entry points are called through the addresses that init() is given, so one
// libkda.so serves both bindings.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "kda.h"

namespace {

struct Failed {};  // a Python error is set

[[noreturn]] void fail(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw Failed{};
}

decltype(&kda_tree_step) p_tree_step;
decltype(&kda_tree_commit) p_tree_commit;
decltype(&kda_tree_conv) p_tree_conv;
decltype(&kda_tree_conv_commit) p_tree_conv_commit;
decltype(&kda_draft_verify) p_draft_verify;
decltype(&kda_linear_prefill) p_linear_prefill;
decltype(&kda_linear_decode_step) p_linear_decode_step;
decltype(&kda_rope) p_rope;

using Shape = std::initializer_list<int64_t>;

std::string text(c10::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " is not a tensor");
    return THPVariable_Unpack(o);
}

// The address of a contiguous device tensor of this type and shape; None passes as null.
void *arg(PyObject *o, c10::ScalarType type, Shape shape, const char *name) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, std::string(name) + " is " + c10::toString(t.scalar_type()) + ", libkda takes " + c10::toString(type) + " here");
    const c10::IntArrayRef want(shape.begin(), shape.size());
    if (t.sizes() != want) fail(PyExc_ValueError, std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(want));
    if (!t.is_cuda()) fail(PyExc_ValueError, "libkda takes device tensors; " + std::string(name) + " is on " + t.device().str());
    if (!t.is_contiguous()) fail(PyExc_ValueError, "libkda takes contiguous tensors; " + std::string(name) + " is not");
    return t.data_ptr();
}
template <typename T>
T *arg(PyObject *o, Shape shape, const char *name) {
    return static_cast<T *>(arg(o, sizeof(T) == 4 && std::is_integral_v<T> ? c10::ScalarType::Int : c10::ScalarType::Float, shape, name));
}

// Sizes of a tensor that others are checked against.
const at::Tensor &lead(PyObject *o, int dims, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != dims) fail(PyExc_ValueError, std::string(name) + " has shape " + text(t.sizes()) + ", expected " + std::to_string(dims) + " dimensions");
    return t;
}
kda_dtype dtype(const at::Tensor &t) {
    if (t.scalar_type() == c10::ScalarType::BFloat16) return KDA_BF16;
    if (t.scalar_type() == c10::ScalarType::Float) return KDA_F32;
    fail(PyExc_TypeError, std::string("libkda takes bf16 or fp32, got ") + c10::toString(t.scalar_type()));
}
int32_t small(int64_t n, const char *name) {
    if (n > INT32_MAX) fail(PyExc_ValueError, std::string(name) + " is too large");
    return (int32_t)n;
}
int32_t integer(PyObject *o, const char *name) {
    const long n = PyLong_AsLong(o);
    if (n == -1 && PyErr_Occurred()) throw Failed{};
    if (n > INT32_MAX || n < INT32_MIN) fail(PyExc_ValueError, std::string(name) + " is out of range");
    return (int32_t)n;
}
float real(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Failed{};
    return (float)x;
}
bool truth(PyObject *o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw Failed{};
    return t != 0;
}
// The given torch.cuda.Stream, or the current one of the tensor's device.
void *stream_of(PyObject *stream, const at::Tensor &t) {
    if (stream == Py_None) return t.is_cuda() ? c10::cuda::getCurrentCUDAStream(t.device().index()).stream() : nullptr;
    PyObject *s = PyObject_GetAttrString(stream, "cuda_stream");
    if (!s) throw Failed{};
    void *p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw Failed{};
    return p;
}

// The device of a call's tensors: a launch goes to the current device, so they have to share one and it has to be made
// current.  (Tensors on the host are refused where they are read.)
std::optional<c10::Device> device_of(PyObject *const *a, Py_ssize_t n) {
    std::optional<c10::Device> device;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!THPVariable_Check(a[i])) continue;
        const c10::Device here = THPVariable_Unpack(a[i]).device();
        if (!here.is_cuda()) continue;
        if (device && *device != here) fail(PyExc_ValueError, "libkda takes tensors of one device; got " + device->str() + " and " + here.str());
        device = here;
    }
    return device;
}

// Runs a call's body on its tensors' device; errors of any kind become Python's.
template <typename F>
PyObject *guarded(PyObject *const *a, Py_ssize_t got, Py_ssize_t want, F body) {
    try {
        if (got != want) fail(PyExc_TypeError, "wrong number of arguments");
        const c10::cuda::OptionalCUDAGuard guard(device_of(a, got));
        return PyLong_FromLong(body());
    } catch (const Failed &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// q, k, v, g, beta, parent, cu_nodes, seq_idx, S_pool, o, u, max_nodes, status, stream, qk_l2norm, qk_eps, out_gate,
// out_weight, out_eps
PyObject *tree_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, 19, [&] {
        const at::Tensor &q = lead(a[0], 3, "q"), &cu = lead(a[6], 1, "cu_nodes"), &pool = lead(a[8], 4, "S_pool");
        const kda_dtype dt = dtype(q);
        const auto type = q.scalar_type();
        const int64_t T = q.size(0), H = q.size(1), d = q.size(2), N = cu.size(0) - 1, slots = pool.size(0);
        kda_fusion_opts opts{truth(a[14]), real(a[15]), arg(a[16], type, {T, H, d}, "out_gate"), arg<float>(a[17], {d}, "out_weight"), real(a[18])};
        return (long)p_tree_step(arg(a[0], type, {T, H, d}, "q"), arg(a[1], type, {T, H, d}, "k"), arg(a[2], type, {T, H, d}, "v"),
                                 arg<float>(a[3], {T, H, d}, "g"), arg<float>(a[4], {T, H}, "beta"), arg<int32_t>(a[5], {T}, "parent"),
                                 arg<int32_t>(a[6], {N + 1}, "cu_nodes"), arg<int32_t>(a[7], {N}, "seq_idx"), small(N, "the batch"),
                                 small(T, "the number of nodes"), integer(a[11], "max_nodes"), small(slots, "the pool"), small(H, "H"),
                                 small(d, "d"), small(d, "d"), dt, arg<float>(a[8], {slots, H, d, d}, "S_pool"),
                                 arg(a[9], type, {T, H, d}, "o"), arg<float>(a[10], {T, H, d}, "u"), arg<int32_t>(a[12], {1}, "status"),
                                 stream_of(a[13], q), opts.qk_l2norm || opts.out_gate ? &opts : nullptr);
    });
}

// k, g, u, cu_nodes, path, path_len, seq_idx, S_pool, status, stream, qk_l2norm, qk_eps
PyObject *tree_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, 12, [&] {
        const at::Tensor &k = lead(a[0], 3, "k"), &cu = lead(a[3], 1, "cu_nodes"), &path = lead(a[4], 2, "path"), &pool = lead(a[7], 4, "S_pool");
        const kda_dtype dt = dtype(k);
        const int64_t T = k.size(0), H = k.size(1), d = k.size(2), N = cu.size(0) - 1, slots = pool.size(0), width = path.size(1);
        kda_fusion_opts opts{truth(a[10]), real(a[11]), nullptr, nullptr, 0.f};
        return (long)p_tree_commit(arg(a[0], k.scalar_type(), {T, H, d}, "k"), arg<float>(a[1], {T, H, d}, "g"), arg<float>(a[2], {T, H, d}, "u"),
                                   arg<int32_t>(a[3], {N + 1}, "cu_nodes"), arg<int32_t>(a[4], {N, width}, "path"),
                                   arg<int32_t>(a[5], {N}, "path_len"), arg<int32_t>(a[6], {N}, "seq_idx"), small(N, "the batch"),
                                   small(T, "the number of nodes"), small(width, "the path"), small(slots, "the pool"), small(H, "H"),
                                   small(d, "d"), small(d, "d"), dt, arg<float>(a[7], {slots, H, d, d}, "S_pool"),
                                   arg<int32_t>(a[8], {1}, "status"), stream_of(a[9], k), opts.qk_l2norm ? &opts : nullptr);
    });
}

// x, w, parent, cu_nodes, seq_idx, conv_pool, y, max_nodes, status, stream
PyObject *tree_conv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, 10, [&] {
        const at::Tensor &x = lead(a[0], 2, "x"), &w = lead(a[1], 2, "w"), &cu = lead(a[3], 1, "cu_nodes"), &pool = lead(a[5], 3, "conv_pool");
        const kda_dtype dt = dtype(x);
        const int64_t T = x.size(0), C = x.size(1), W = w.size(1), N = cu.size(0) - 1, slots = pool.size(0);
        return (long)p_tree_conv(arg(a[0], x.scalar_type(), {T, C}, "x"), arg<float>(a[1], {C, W}, "w"), arg<int32_t>(a[2], {T}, "parent"),
                                 arg<int32_t>(a[3], {N + 1}, "cu_nodes"), arg<int32_t>(a[4], {N}, "seq_idx"), small(N, "the batch"),
                                 small(T, "the number of nodes"), integer(a[7], "max_nodes"), small(slots, "the pool"), small(C, "C"),
                                 small(W, "W"), dt, arg<float>(a[5], {slots, W - 1, C}, "conv_pool"), arg(a[6], x.scalar_type(), {T, C}, "y"),
                                 arg<int32_t>(a[8], {1}, "status"), stream_of(a[9], x));
    });
}

// x, cu_nodes, path, path_len, seq_idx, conv_pool, status, stream
PyObject *tree_conv_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, 8, [&] {
        const at::Tensor &x = lead(a[0], 2, "x"), &cu = lead(a[1], 1, "cu_nodes"), &path = lead(a[2], 2, "path"), &pool = lead(a[5], 3, "conv_pool");
        const kda_dtype dt = dtype(x);
        const int64_t T = x.size(0), C = x.size(1), N = cu.size(0) - 1, slots = pool.size(0), carried = pool.size(1), width = path.size(1);
        return (long)p_tree_conv_commit(arg(a[0], x.scalar_type(), {T, C}, "x"), arg<int32_t>(a[1], {N + 1}, "cu_nodes"),
                                        arg<int32_t>(a[2], {N, width}, "path"), arg<int32_t>(a[3], {N}, "path_len"),
                                        arg<int32_t>(a[4], {N}, "seq_idx"), small(N, "the batch"), small(T, "the number of nodes"),
                                        small(width, "the path"), small(slots, "the pool"), small(C, "C"), small(carried + 1, "W"), dt,
                                        arg<float>(a[5], {slots, carried, C}, "conv_pool"), arg<int32_t>(a[6], {1}, "status"),
                                        stream_of(a[7], x));
    });
}

// logits, tokens, parent, cu_nodes, u_accept, u_next, path, path_len, next_token, draft_probs, temperature, status, stream
PyObject *draft_verify(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, 13, [&] {
        const at::Tensor &l = lead(a[0], 2, "logits"), &cu = lead(a[3], 1, "cu_nodes"), &path = lead(a[6], 2, "path");
        const kda_dtype dt = dtype(l);
        const int64_t T = l.size(0), V = l.size(1), N = cu.size(0) - 1, width = path.size(1);
        return (long)p_draft_verify(arg(a[0], l.scalar_type(), {T, V}, "logits"), arg<float>(a[9], {T, V}, "draft_probs"),
                                    arg<int32_t>(a[1], {T}, "tokens"), arg<int32_t>(a[2], {T}, "parent"),
                                    arg<int32_t>(a[3], {N + 1}, "cu_nodes"), arg<float>(a[10], {N}, "temperature"),
                                    arg<float>(a[4], {T}, "u_accept"), arg<float>(a[5], {N}, "u_next"), small(N, "the batch"),
                                    small(T, "the number of nodes"), small(V, "V"), dt, small(width, "the path"),
                                    arg<int32_t>(a[6], {N, width}, "path"), arg<int32_t>(a[7], {N}, "path_len"),
                                    arg<int32_t>(a[8], {N}, "next_token"), arg<int32_t>(a[11], {1}, "status"), stream_of(a[12], l));
    });
}

// A linear-attention call's sizes, from its q [rows, H_qk, d] and v [rows, H, d].
struct LinearSizes {
    const at::Tensor &q, &v;
    int64_t rows, H, Hqk, d;
    c10::ScalarType type;
    bool per_token;
};
LinearSizes linear_sizes(PyObject *oq, PyObject *ov, PyObject *og) {
    const at::Tensor &q = lead(oq, 3, "q"), &v = lead(ov, 3, "v"), &g = tensor(og, "g");
    dtype(q);
    if (g.dim() != 1 && g.dim() != 2) fail(PyExc_ValueError, "g has shape " + text(g.sizes()) + ", expected one log-decay a token and head, or one a head");
    return {q, v, v.size(0), v.size(1), q.size(1), v.size(2), q.scalar_type(), g.dim() == 2};
}
float *decays(PyObject *o, const LinearSizes &s) {
    return s.per_token ? arg<float>(o, {s.rows, s.H}, "g") : arg<float>(o, {s.H}, "g");
}

// q, k, v, g, cu_seqlens, o, S0, S_final, workspace, stream, qk_l2norm, qk_eps, out_gate, out_weight, out_eps
PyObject *linear_prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, 15, [&] {
        const LinearSizes s = linear_sizes(a[0], a[2], a[3]);
        const at::Tensor &cu = lead(a[4], 1, "cu_seqlens"), &ws = lead(a[8], 1, "workspace");
        const int64_t N = cu.size(0) - 1;
        kda_fusion_opts opts{truth(a[10]), real(a[11]), arg(a[12], s.type, {s.rows, s.H, s.d}, "out_gate"), arg<float>(a[13], {s.d}, "out_weight"), real(a[14])};
        return (long)p_linear_prefill(arg(a[0], s.type, {s.rows, s.Hqk, s.d}, "q"), arg(a[1], s.type, {s.rows, s.Hqk, s.d}, "k"),
                                      arg(a[2], s.type, {s.rows, s.H, s.d}, "v"), decays(a[3], s), s.per_token,
                                      arg<int32_t>(a[4], {N + 1}, "cu_seqlens"), small(N, "the batch"), small(s.rows, "the number of tokens"),
                                      small(s.H, "H"), small(s.Hqk, "H_qk"), small(s.d, "d"), small(s.d, "d"), dtype(s.q),
                                      arg<float>(a[6], {N, s.H, s.d, s.d}, "S0"), arg(a[5], s.type, {s.rows, s.H, s.d}, "o"),
                                      arg<float>(a[7], {N, s.H, s.d, s.d}, "S_final"), arg(a[8], c10::ScalarType::Byte, {ws.size(0)}, "workspace"),
                                      (size_t)ws.size(0), stream_of(a[9], s.q), opts.qk_l2norm || opts.out_gate ? &opts : nullptr);
    });
}

// q, k, v, g, S_pool, o, seq_idx, status, stream, qk_l2norm, qk_eps, out_gate, out_weight, out_eps
PyObject *linear_decode_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, 14, [&] {
        const LinearSizes s = linear_sizes(a[0], a[2], a[3]);
        const at::Tensor &pool = lead(a[4], 4, "S_pool");
        const int64_t slots = pool.size(0);
        if (a[6] == Py_None && slots < s.rows) fail(PyExc_ValueError, "S_pool has fewer slots than there are sequences");
        kda_fusion_opts opts{truth(a[9]), real(a[10]), arg(a[11], s.type, {s.rows, s.H, s.d}, "out_gate"), arg<float>(a[12], {s.d}, "out_weight"), real(a[13])};
        return (long)p_linear_decode_step(arg(a[0], s.type, {s.rows, s.Hqk, s.d}, "q"), arg(a[1], s.type, {s.rows, s.Hqk, s.d}, "k"),
                                          arg(a[2], s.type, {s.rows, s.H, s.d}, "v"), decays(a[3], s), s.per_token,
                                          arg<int32_t>(a[6], {s.rows}, "seq_idx"), small(s.rows, "the batch"), small(slots, "the pool"),
                                          small(s.H, "H"), small(s.Hqk, "H_qk"), small(s.d, "d"), small(s.d, "d"), dtype(s.q),
                                          arg<float>(a[4], {slots, s.H, s.d, s.d}, "S_pool"), arg(a[5], s.type, {s.rows, s.H, s.d}, "o"),
                                          arg<int32_t>(a[7], {1}, "status"), stream_of(a[8], s.q), opts.qk_l2norm || opts.out_gate ? &opts : nullptr);
    });
}

// q, k, positions, steps, q_out, k_out, interleaved, scale, stream
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, 9, [&] {
        const at::Tensor &q = lead(a[0], 3, "q"), &steps = lead(a[3], 1, "steps");
        const kda_dtype dt = dtype(q);
        const auto type = q.scalar_type();
        const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), Hk = a[1] == Py_None ? 0 : lead(a[1], 3, "k").size(1);
        if (Hk == 0 && a[5] != Py_None && a[1] == Py_None) fail(PyExc_ValueError, "k_out without k");
        return (long)p_rope(arg(a[0], type, {T, Hq, d}, "q"), arg(a[1], type, {T, Hk, d}, "k"), arg<int32_t>(a[2], {T}, "positions"),
                            static_cast<const uint64_t *>(arg(a[3], c10::ScalarType::Long, {steps.size(0)}, "steps")), small(T, "the number of tokens"),
                            small(Hq, "H_q"), small(Hk, "H_k"), small(d, "d"), small(2 * steps.size(0), "rot"), truth(a[6]), real(a[7]), dt,
                            arg(a[4], type, {T, Hq, d}, "q_out"), arg(a[5], type, {T, Hk, d}, "k_out"), stream_of(a[8], q));
    });
}

// The addresses of the entry points, in the order of the functions above.
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[8];
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "init takes eight addresses");
        return nullptr;
    }
    for (int i = 0; i < 8; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    p_tree_step = reinterpret_cast<decltype(p_tree_step)>(p[0]);
    p_tree_commit = reinterpret_cast<decltype(p_tree_commit)>(p[1]);
    p_tree_conv = reinterpret_cast<decltype(p_tree_conv)>(p[2]);
    p_tree_conv_commit = reinterpret_cast<decltype(p_tree_conv_commit)>(p[3]);
    p_draft_verify = reinterpret_cast<decltype(p_draft_verify)>(p[4]);
    p_linear_prefill = reinterpret_cast<decltype(p_linear_prefill)>(p[5]);
    p_linear_decode_step = reinterpret_cast<decltype(p_linear_decode_step)>(p[6]);
    p_rope = reinterpret_cast<decltype(p_rope)>(p[7]);
    Py_RETURN_NONE;
}

#define KDA_FUNCTION(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef functions[] = {KDA_FUNCTION(init),             KDA_FUNCTION(tree_step),    KDA_FUNCTION(tree_commit), KDA_FUNCTION(tree_conv),
                           KDA_FUNCTION(tree_conv_commit), KDA_FUNCTION(draft_verify),
                           KDA_FUNCTION(linear_prefill),   KDA_FUNCTION(linear_decode_step), KDA_FUNCTION(rope), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_tree", nullptr, -1, functions, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_tree() { return PyModule_Create(&module); }
