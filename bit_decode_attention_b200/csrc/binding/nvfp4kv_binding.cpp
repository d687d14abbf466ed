// nvfp4kv_binding.cpp -- argument marshalling of the tree-step entry points for
// the Python package (extension module `_binding`).
//
// A decoding step calls these entry points once or more per layer with fifteen
// to twenty-five tensors each, and their kernels take a few microseconds:
// checking every tensor from Python and passing it through ctypes took 10 to
// 19 us a call, longer than the kernels.  Here the same checks take about 1 us.
// The functions check shapes, types, contiguity and devices, fill the plane
// structs, call the C ABI and return its status; nothing is computed or kept.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdio>
#include <exception>
#include <initializer_list>
#include <string>

#include "nvfp4kv.h"

namespace {

struct Failed {};                                     // a Python exception is set

[[noreturn]] void fail(PyObject* type, const std::string& text) {
    PyErr_SetString(type, text.c_str());
    throw Failed{};
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const at::Tensor& tensor_of(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// o as a contiguous tensor of this type and shape on CUDA device `cur`
void* need(PyObject* o, int cur, at::ScalarType type, at::IntArrayRef shape, const char* name) {
    const at::Tensor& t = tensor_of(o, name);
    if (t.get_device() != cur || t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        fail(PyExc_ValueError, std::string(name) + " must be a contiguous CUDA tensor " + shape_text(shape) + " of " +
                                   c10::toString(type) + " on the current device (" + std::to_string(cur) + "), got " +
                                   (t.is_contiguous() ? "" : "a non-contiguous ") + shape_text(t.sizes()) + " of " +
                                   c10::toString(t.scalar_type()) + " on " + t.device().str());
    return t.data_ptr();
}

void* need_or_null(PyObject* o, int cur, at::ScalarType type, at::IntArrayRef shape, const char* name) {
    return o == Py_None ? nullptr : need(o, cur, type, shape, name);
}

int32_t* ints(PyObject* o, int cur, at::IntArrayRef shape, const char* name) {
    return static_cast<int32_t*>(need(o, cur, at::kInt, shape, name));
}

int32_t* ints_or_null(PyObject* o, int cur, at::IntArrayRef shape, const char* name) {
    return o == Py_None ? nullptr : ints(o, cur, shape, name);
}

// a tensor scale or the status word: one element, on the device
void* scalar(PyObject* o, int cur, at::ScalarType type, const char* name) {
    const at::Tensor& t = tensor_of(o, name);
    if (t.get_device() != cur || t.scalar_type() != type || t.numel() < 1)
        fail(PyExc_ValueError, std::string(name) + " must be a CUDA tensor of one " + c10::toString(type) +
                                   " on the current device (" + std::to_string(cur) + ")");
    return t.data_ptr();
}

int32_t* status_word(PyObject* o, int cur) {
    return o == Py_None ? nullptr : static_cast<int32_t*>(scalar(o, cur, at::kInt, "status"));
}

nvfp4_dtype dtype_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return NVFP4_IN_BF16;
    if (t.scalar_type() == at::kFloat) return NVFP4_IN_F32;
    fail(PyExc_TypeError, std::string("inputs must be bfloat16 or float32, got ") + c10::toString(t.scalar_type()));
}

PyObject *s_codes, *s_scales, *s_block_table;

struct Ref {
    PyObject* o;
    explicit Ref(PyObject* p) : o(p) {
        if (o == nullptr) throw Failed{};
    }
    Ref(const Ref&) = delete;
    ~Ref() { Py_DECREF(o); }
};

int32_t narrow(int64_t v) {
    if (v > INT32_MAX) fail(PyExc_ValueError, "a plane's dimension does not fit 32 bits");
    return (int32_t)v;
}

struct Dims {
    int64_t B, H, D;
};

// codes [n][H][S][D/2] and scales [n][H][S][D/16] of a plane
std::array<int64_t, 4> code_shape(PyObject* plane, int cur, uint8_t*& codes, uint8_t*& scales) {
    const Ref c(PyObject_GetAttr(plane, s_codes)), s(PyObject_GetAttr(plane, s_scales));
    const at::Tensor& t = tensor_of(c.o, "codes");
    if (t.dim() != 4) fail(PyExc_ValueError, "codes must have four dimensions");
    const std::array<int64_t, 4> n{t.size(0), t.size(1), t.size(2), t.size(3)};
    codes = static_cast<uint8_t*>(need(c.o, cur, at::kByte, n, "codes"));
    scales = static_cast<uint8_t*>(need(s.o, cur, at::kByte, {n[0], n[1], n[2], n[3] / 8}, "scales"));
    return n;
}

Dims fill(PyObject* plane, int cur, nvfp4_kv_plane& out) {
    const auto n = code_shape(plane, cur, out.codes, out.scales);
    out.B = narrow(n[0]);
    out.H_kv = narrow(n[1]);
    out.S_max = narrow(n[2]);
    out.D = narrow(2 * n[3]);
    return {n[0], n[1], 2 * n[3]};
}

Dims fill(PyObject* plane, int cur, nvfp4_kv_paged_plane& out) {
    const auto n = code_shape(plane, cur, out.codes, out.scales);
    const Ref b(PyObject_GetAttr(plane, s_block_table));
    const at::Tensor& t = tensor_of(b.o, "block_table");
    if (t.dim() != 2) fail(PyExc_ValueError, "block_table must have two dimensions");
    out.block_table = ints(b.o, cur, t.sizes(), "block_table");
    out.num_pages = narrow(n[0]);
    out.H_kv = narrow(n[1]);
    out.page_tokens = narrow(n[2]);
    out.D = narrow(2 * n[3]);
    out.B = narrow(t.size(0));
    out.max_pages = narrow(t.size(1));
    return {t.size(0), n[1], 2 * n[3]};
}

template <class Plane>
struct Cache {
    Plane k, v;
    Dims d;
    Cache(PyObject* pk, PyObject* pv, int cur) : k{}, v{}, d(fill(pk, cur, k)) { fill(pv, cur, v); }
};

// elements between tokens of x [B][n][H][D]: dense heads, evenly spaced tokens
// (a slice of a packed projection has them; a tensor expanded over tokens or sequences has not)
const void* rows(PyObject* o, int cur, at::ScalarType type, int64_t B, int64_t n, int64_t H, int64_t D, const char* name,
                 int64_t& step) {
    const at::Tensor& t = tensor_of(o, name);
    if (t.get_device() != cur || t.scalar_type() != type || t.sizes() != at::IntArrayRef({B, n, H, D}))
        fail(PyExc_ValueError, std::string(name) + " must be a CUDA tensor " + shape_text({B, n, H, D}) + " of " +
                                   c10::toString(type) + " on the current device (" + std::to_string(cur) + "), got " +
                                   shape_text(t.sizes()) + " of " + c10::toString(t.scalar_type()) + " on " +
                                   t.device().str());
    step = H * D;
    if (t.numel() == 0) return t.data_ptr();
    const auto s = t.strides();
    step = n > 1 ? s[1] : (B > 1 ? s[0] : H * D);
    // a step below a token's row is a broadcast (0, which the C call takes for dense) or an overlap
    if ((D > 1 && s[3] != 1) || (H > 1 && s[2] != D) || (B > 1 && n > 1 && s[0] != n * s[1]) ||
        (B * n > 1 && step < H * D))
        fail(PyExc_ValueError, std::string(name) + " must have dense heads and evenly spaced tokens");
    return t.data_ptr();
}

long as_long(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Failed{};
    return v;
}

bool as_bool(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Failed{};
    return v != 0;
}

float as_float(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Failed{};
    return (float)v;
}

nvfp4_stream_t as_stream(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw Failed{};
    return static_cast<nvfp4_stream_t>(p);
}

void dims_of(const at::Tensor& t, int64_t n, const char* name) {
    if (t.dim() != n) fail(PyExc_ValueError, std::string(name) + " must have " + std::to_string(n) + " dimensions");
}

// (device, stream, paged, x_q, x_k, x_v, start_pos, s_tensor_k, s_tensor_v, k, v, w_q, w_k, eps, rope_table,
//  interleaved, positions, n_valid, q_out, new_lens, status)
template <class Plane, class F>
int norm_rope(PyObject* const* a, int cur, F call) {
    const Cache<Plane> c(a[9], a[10], cur);
    const at::Tensor& xq = tensor_of(a[3], "x_q");
    dims_of(xq, 4, "x_q");
    const nvfp4_dtype dt = dtype_of(xq);
    const at::ScalarType type = xq.scalar_type();
    const int64_t B = c.d.B, D = c.d.D, n = xq.size(1), Hq = xq.size(2);
    int64_t sq, sk, sv;
    const void* q = rows(a[3], cur, type, B, n, Hq, D, "x_q", sq);
    const void* k = rows(a[4], cur, type, B, n, c.d.H, D, "x_k", sk);
    const void* v = rows(a[5], cur, type, B, n, c.d.H, D, "x_v", sv);
    const float* table = nullptr;
    int64_t P = 0, R = 0;
    if (a[14] != Py_None) {
        const at::Tensor& t = tensor_of(a[14], "rope_table");
        dims_of(t, 2, "rope_table");
        P = t.size(0);
        R = t.size(1);
        table = static_cast<const float*>(need(a[14], cur, at::kFloat, {P, R}, "rope_table"));
    }
    return call(q, k, v, dt, narrow(n), narrow(Hq), sq, sk, sv, need_or_null(a[11], cur, type, {D}, "w_q"),
                need_or_null(a[12], cur, type, {D}, "w_k"), as_float(a[13]), table, narrow(P), narrow(R),
                as_bool(a[15]), ints_or_null(a[16], cur, {B, n}, "positions"),
                ints(a[6], cur, {B}, "start_pos"), ints_or_null(a[17], cur, {B}, "n_valid"),
                ints_or_null(a[19], cur, {B}, "new_lens"),
                static_cast<const float*>(scalar(a[7], cur, at::kFloat, "s_tensor_k")),
                static_cast<const float*>(scalar(a[8], cur, at::kFloat, "s_tensor_v")), &c.k, &c.v,
                need(a[18], cur, type, {B, n, Hq, D}, "q_out"), status_word(a[20], cur), as_stream(a[1]));
}

// (device, stream, paged, q, k, v, s_tensor_k, s_tensor_v, start_pos, tree_mask, n_nodes, softmax_scale, out,
//  workspace, status)
template <class Plane, class F>
int tree(PyObject* const* a, int cur, F call) {
    const Cache<Plane> c(a[4], a[5], cur);
    const at::Tensor& q = tensor_of(a[3], "q");
    dims_of(q, 4, "q");
    const int64_t B = c.d.B, D = c.d.D, N = q.size(1), Hq = q.size(2), W = (N + 31) / 32;
    const int32_t* mask = nullptr;
    int64_t stride = 0;
    if (a[9] != Py_None) {
        const bool each = tensor_of(a[9], "tree_mask").dim() == 3;
        stride = each ? N * W : 0;
        mask = each ? ints(a[9], cur, {B, N, W}, "tree_mask") : ints(a[9], cur, {N, W}, "tree_mask");
    }
    const at::Tensor& out = tensor_of(a[12], "out");
    const at::Tensor& ws = tensor_of(a[13], "workspace");
    if (ws.get_device() != cur || !ws.is_contiguous())
        fail(PyExc_ValueError, "workspace must be a contiguous tensor on the current CUDA device");
    return call(need(a[3], cur, q.scalar_type(), {B, N, Hq, D}, "q"), dtype_of(q), narrow(N), narrow(Hq), &c.k, &c.v,
                static_cast<const float*>(scalar(a[6], cur, at::kFloat, "s_tensor_k")),
                static_cast<const float*>(scalar(a[7], cur, at::kFloat, "s_tensor_v")),
                ints(a[8], cur, {B}, "start_pos"), ints_or_null(a[10], cur, {B}, "n_nodes"), mask, stride,
                as_float(a[11]), need(a[12], cur, out.scalar_type(), {B, N, Hq, D}, "out"), dtype_of(out),
                ws.data_ptr(), (size_t)ws.nbytes(), status_word(a[14], cur), as_stream(a[1]));
}

// (device, stream, target_probs, draft_probs, tokens, parents, u_accept, u_sample, n_nodes, path, n_accepted,
//  next_token, status)
int verify(PyObject* const* a, int cur) {
    const at::Tensor& p = tensor_of(a[2], "target_probs");
    dims_of(p, 3, "target_probs");
    const int64_t B = p.size(0), N = p.size(1), V = p.size(2);
    const at::ScalarType type = p.scalar_type();
    const bool shared = tensor_of(a[5], "parents").dim() == 1;
    return nvfp4_verify_drafts(
        need(a[2], cur, type, {B, N, V}, "target_probs"), need_or_null(a[3], cur, type, {B, N, V}, "draft_probs"),
        dtype_of(p), narrow(B), narrow(N), narrow(V), ints(a[4], cur, {B, N}, "tokens"),
        shared ? ints(a[5], cur, {N}, "parents") : ints(a[5], cur, {B, N}, "parents"), shared,
        static_cast<const float*>(need(a[6], cur, at::kFloat, {B, N}, "u_accept")),
        static_cast<const float*>(need(a[7], cur, at::kFloat, {B}, "u_sample")),
        ints_or_null(a[8], cur, {B}, "n_nodes"), ints(a[9], cur, {B, N}, "path"),
        ints(a[10], cur, {B}, "n_accepted"), ints(a[11], cur, {B}, "next_token"), status_word(a[12], cur),
        as_stream(a[1]));
}

// (device, stream, paged, address of the plane structs, planes, B, start_pos, path, n_accepted, new_lens, status)
template <class Plane, class F>
int commit(PyObject* const* a, int cur, F call) {
    const auto* planes = static_cast<const Plane*>(PyLong_AsVoidPtr(a[3]));
    if (planes == nullptr && PyErr_Occurred()) throw Failed{};
    const int64_t B = as_long(a[5]);
    const at::Tensor& path = tensor_of(a[7], "path");
    dims_of(path, 2, "path");
    const int64_t N = path.size(1);
    return call(planes, (int)as_long(a[4]), narrow(N), ints(a[6], cur, {B}, "start_pos"),
                ints(a[7], cur, {B, N}, "path"), ints(a[8], cur, {B}, "n_accepted"),
                ints_or_null(a[9], cur, {B}, "new_lens"), status_word(a[10], cur), as_stream(a[1]));
}

template <class F>
PyObject* entry(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, F f) {
    try {
        if (n != want) fail(PyExc_TypeError, "wrong number of arguments");
        return PyLong_FromLong(f((int)as_long(a[0])));
    } catch (const Failed&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject* py_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(a, n, 21, [&](int cur) {
        return as_bool(a[2]) ? norm_rope<nvfp4_kv_paged_plane>(a, cur, nvfp4_qk_norm_rope_append_paged)
                                     : norm_rope<nvfp4_kv_plane>(a, cur, nvfp4_qk_norm_rope_append);
    });
}

PyObject* py_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(a, n, 15, [&](int cur) {
        return as_bool(a[2]) ? tree<nvfp4_kv_paged_plane>(a, cur, nvfp4_tree_attention_paged)
                                     : tree<nvfp4_kv_plane>(a, cur, nvfp4_tree_attention);
    });
}

PyObject* py_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(a, n, 13, [&](int cur) { return verify(a, cur); });
}

PyObject* py_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(a, n, 11, [&](int cur) {
        return as_bool(a[2]) ? commit<nvfp4_kv_paged_plane>(a, cur, nvfp4_kv_commit_path_paged)
                                     : commit<nvfp4_kv_plane>(a, cur, nvfp4_kv_commit_path);
    });
}

// (device, paged, planes) -> (bytes of the plane structs, B)
PyObject* py_planes(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        if (n != 3) fail(PyExc_TypeError, "wrong number of arguments");
        const int cur = (int)as_long(a[0]);
        const bool paged = as_bool(a[1]);
        const Ref seq(PySequence_Fast(a[2], "planes must be a sequence"));
        const Py_ssize_t m = PySequence_Fast_GET_SIZE(seq.o);
        std::string bytes;
        int64_t B = 0;
        for (Py_ssize_t i = 0; i < m; ++i) {
            PyObject* p = PySequence_Fast_GET_ITEM(seq.o, i);
            if (paged) {
                nvfp4_kv_paged_plane s{};
                B = fill(p, cur, s).B;
                bytes.append(reinterpret_cast<const char*>(&s), sizeof(s));
            } else {
                nvfp4_kv_plane s{};
                B = fill(p, cur, s).B;
                bytes.append(reinterpret_cast<const char*>(&s), sizeof(s));
            }
        }
        return Py_BuildValue("(y#L)", bytes.data(), (Py_ssize_t)bytes.size(), (long long)B);
    } catch (const Failed&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define NVFP4_FAST(NAME, FN) {NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(FN)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    NVFP4_FAST("qk_norm_rope_append", py_norm_rope), NVFP4_FAST("tree_attention", py_tree),
    NVFP4_FAST("verify_drafts", py_verify),          NVFP4_FAST("commit_path", py_commit),
    NVFP4_FAST("planes", py_planes),                 {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    s_codes = PyUnicode_InternFromString("codes");
    s_scales = PyUnicode_InternFromString("scales");
    s_block_table = PyUnicode_InternFromString("block_table");
    if (s_codes == nullptr || s_scales == nullptr || s_block_table == nullptr) return nullptr;
    PyObject* const m = PyModule_Create(&module);
    // the build looks for this text, to tell a module that was built against another torch
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", NVFP4_BINDING_STAMP) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
