// Argument checks and calls of the operators around and between the linears, for the Python
// binding: a Python module of its own (_lib/rudder_bind.so).
//
// Their smallest calls take the GPU 3 to 6 us, and checking seven to nine
// tensors in Python and converting two dozen arguments took as long (K = N =
// 2048, one row: 6.0 us a call, now 4.4).  Tensors are checked for their type,
// layout, place and size against the sizes passed; device addresses (ints)
// pass through unchecked, None is a null pointer.  The first argument of every
// call is the number of the current device, where all tensors have to lie.
#include <Python.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "rudder.h"
#include "rudder_attention.h"
#include "rudder_block.h"

namespace {

// The entry points, from the library that the binding has loaded.
struct Library {
    decltype(&rudder_quantize_weights_grouped) quantize_weights_grouped;
    decltype(&rudder_matvec_w4) matvec_w4;
    decltype(&rudder_grouped_weight_bytes) grouped_weight_bytes;
    decltype(&rudder_grouped_scale_count) grouped_scale_count;
    decltype(&rudder_cache_append) cache_append;
    decltype(&rudder_cache_dequant) cache_dequant;
    decltype(&rudder_cache_attention) cache_attention;
    decltype(&rudder_cross_attention) cross_attention;
    decltype(&rudder_packed_act_bytes) packed_act_bytes;
    decltype(&rudder_norm) norm;
    decltype(&rudder_norm_quant) norm_quant;
    decltype(&rudder_dequant_act) dequant_act;
    decltype(&rudder_rotary) rotary;
    decltype(&rudder_prompt_attention) prompt_attention;
} lib = {};

struct Failure {};                                 // a Python error is set

[[noreturn]] void refuse(const char* name, PyObject* o, const char* why, long long least,
                         const char* what) {
    PyObject* dtype = PyObject_GetAttrString(o, "dtype");
    PyObject* shape = dtype ? PyObject_GetAttrString(o, "shape") : nullptr;
    PyObject* strides = shape ? PyObject_CallMethod(o, "stride", nullptr) : nullptr;
    if (strides)
        PyErr_Format(PyExc_ValueError, "%s: %S, %S, strides %S: %s%lld %s", name, dtype, shape,
                     strides, why, least, what);
    Py_XDECREF(dtype);
    Py_XDECREF(shape);
    Py_XDECREF(strides);
    throw Failure{};
}

// The arguments of a call, taken from left to right.
class Args {
  public:
    Args(const char* call, PyObject* const* args, Py_ssize_t n, Py_ssize_t expected)
        : args_(args) {
        if (n == expected && lib.matvec_w4) {
            device_ = integer();
            return;
        }
        PyErr_Format(PyExc_TypeError, "%s: %zd arguments, expected %zd%s", call, n, expected,
                     lib.matvec_w4 ? "" : " (and a library)");
        throw Failure{};
    }

    PyObject* next() { return args_[at_++]; }

    int integer() {
        const long v = PyLong_AsLong(next());
        if (v == -1 && PyErr_Occurred()) throw Failure{};
        if (v != (int)v) {
            PyErr_Format(PyExc_OverflowError, "argument %zd: %ld is no 32-bit integer", at_, v);
            throw Failure{};
        }
        return (int)v;
    }

    float real() {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw Failure{};
        return (float)v;
    }

    int truth() {
        const int v = PyObject_IsTrue(next());
        if (v < 0) throw Failure{};
        return v;
    }

    void* address(PyObject* o) {
        void* p = PyLong_AsVoidPtr(o);
        if (!p && PyErr_Occurred()) throw Failure{};
        return p;
    }

    void* stream() {
        PyObject* o = next();
        return o == Py_None ? nullptr : address(o);
    }

    // A tensor's memory on the current device.
    void* place(const char* name, const at::Tensor& t) {
        if (t.is_cuda() && t.get_device() == device_) return t.data_ptr();
        if (t.is_cuda())
            PyErr_Format(PyExc_ValueError, "%s: on cuda:%d, but the current device is cuda:%d",
                         name, (int)t.get_device(), device_);
        else
            PyErr_Format(PyExc_ValueError, "%s: not on a GPU", name);
        throw Failure{};
    }

  private:
    int device_ = -1;
    PyObject* const* args_;
    Py_ssize_t at_ = 0;
};

bool is(const at::Tensor& t, at::ScalarType type) {
    const at::ScalarType s = t.scalar_type();
    return s == type || (type == at::kBFloat16 && (s == at::kShort || s == at::kUInt16));
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (THPVariable_Check(o)) return THPVariable_Unpack(o);
    PyErr_Format(PyExc_TypeError, "%s: a tensor, an address or None expected", name);
    throw Failure{};
}

// A contiguous tensor of a type with at least that many elements.
template <class T>
T* array(Args& a, const char* name, PyObject* o, at::ScalarType type, long long least) {
    if (o == Py_None) return nullptr;
    if (PyLong_Check(o)) return static_cast<T*>(a.address(o));
    const at::Tensor& t = tensor(name, o);
    if (!is(t, type) || t.numel() < least || !t.is_contiguous())
        refuse(name, o, "expected at least ", least,
               type == at::kBFloat16 ? "contiguous bf16 elements"
               : type == at::kFloat  ? "contiguous fp32 elements"
               : type == at::kDouble ? "contiguous fp64 elements"
               : type == at::kInt    ? "contiguous int32 elements"
               : type == at::kChar   ? "contiguous int8 elements"
                                     : "contiguous uint8 elements");
    return static_cast<T*>(a.place(name, t));
}

// T rows of H heads of D bf16 values: [T, H, D] or [T, H * D], a row's values packed, rows any
// distance apart.  `ld` (None: the tensor's own) is that distance; a single row has none, whatever
// its tensor's stride says.
uint16_t* rows(Args& a, const char* name, PyObject* o, int T, int H, int D, PyObject* distance,
               int& ld) {
    const bool given = distance != Py_None;
    const long want = given ? PyLong_AsLong(distance) : 0;
    if (given && want == -1 && PyErr_Occurred()) throw Failure{};
    const long long width = (long long)H * D;
    long long step = given ? want : width;
    uint16_t* p = nullptr;
    if (o != Py_None && PyLong_Check(o)) {
        p = static_cast<uint16_t*>(a.address(o));
    } else if (o != Py_None) {
        const at::Tensor& t = tensor(name, o);
        bool good = is(t, at::kBFloat16) && (t.dim() == 2 || t.dim() == 3);
        if (good && t.dim() == 3)
            good = t.size(1) == H && t.size(2) == D && t.stride(2) == 1 &&
                   (t.stride(1) == D || H == 1);
        else if (good)
            good = t.size(1) == width && t.stride(1) == 1;
        if (!good || t.size(0) < T || (given && T > 1 && want != t.stride(0)))
            refuse(name, o, "expected at least ", T,
                   "rows of packed bf16 heads, the row distance apart");
        if (T > 1) step = t.stride(0);
        p = static_cast<uint16_t*>(a.place(name, t));
    }
    if (step != (int)step) {
        PyErr_Format(PyExc_OverflowError, "%s: rows %lld elements apart", name, step);
        throw Failure{};
    }
    ld = (int)step;
    return p;
}

// A workspace and its size: a uint8 tensor, or an address that is taken to be large enough.
void* workspace(Args& a, size_t& bytes) {
    PyObject* o = a.next();
    bytes = 0;
    if (o == Py_None) return nullptr;
    bytes = PY_SSIZE_T_MAX;
    if (!PyLong_Check(o)) bytes = (size_t)tensor("workspace", o).numel();
    return array<void>(a, "workspace", o, at::kByte, 0);
}

template <class F>
PyObject* guarded(F f) {
    try {
        return PyLong_FromLong(f());
    } catch (const Failure&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <class F>
int call(F f) {
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f();
    Py_END_ALLOW_THREADS
    return status;
}

long long product(long long a, long long b) { return a > 0 && b > 0 ? a * b : 0; }

// (device, W, K, N, group, Wq, g_scale, stream)
PyObject* quantize_weights_grouped(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_quantize_weights_grouped", args, n, 8);
        PyObject* W = a.next();
        const int K = a.integer(), N = a.integer(), group = a.integer();
        const auto* w = array<uint16_t>(a, "W", W, at::kBFloat16, product(K, N));
        auto* q = array<uint8_t>(a, "Wq", a.next(), at::kByte,
                                 (long long)lib.grouped_weight_bytes(K, N));
        auto* s = array<uint16_t>(a, "g_scale", a.next(), at::kBFloat16,
                                  (long long)lib.grouped_scale_count(K, N, group));
        void* st = a.stream();
        return call([&] { return lib.quantize_weights_grouped(w, K, N, group, q, s, st); });
    });
}

// (device, X, stream_id, Wq, g_scale, comp_a, comp_b, M, N, K, group, S, Y, stream)
PyObject* matvec_w4(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_matvec_w4", args, n, 14);
        PyObject *X = a.next(), *sid = a.next(), *Wq = a.next(), *gs = a.next(), *ca = a.next(),
                 *cb = a.next();
        const int M = a.integer(), N = a.integer(), K = a.integer(), group = a.integer(),
                  S = a.integer();
        PyObject* Y = a.next();
        const auto* x = array<uint16_t>(a, "X", X, at::kBFloat16, product(M, K));
        const auto* st = array<uint8_t>(a, "stream_id", sid, at::kByte, M);
        const auto* q = array<uint8_t>(a, "Wq", Wq, at::kByte,
                                       (long long)lib.grouped_weight_bytes(K, N));
        const auto* s = array<uint16_t>(a, "g_scale", gs, at::kBFloat16,
                                        (long long)lib.grouped_scale_count(K, N, group));
        const auto* fa = array<float>(a, "comp_a", ca, at::kFloat, product(S, N));
        const auto* fb = array<float>(a, "comp_b", cb, at::kFloat, product(S, N));
        auto* y = array<uint16_t>(a, "Y", Y, at::kBFloat16, product(M, N));
        void* stream = a.stream();
        return call([&] {
            return lib.matvec_w4(x, st, q, s, fa, fb, M, N, K, group, S, y, stream);
        });
    });
}

struct Cache {
    PyObject *codes, *scales;
    int8_t* c = nullptr;
    float* s = nullptr;
    void check(Args& a, int num_pages, int Hkv, int D) {
        const long long blocks = product(product(num_pages, Hkv), 2);
        c = array<int8_t>(a, "codes", codes, at::kChar,
                          product(blocks, product(RUDDER_CACHE_PAGE, D)));
        s = array<float>(a, "scales", scales, at::kFloat, blocks);
    }
};

// (device, K, V, row_start, pos, page_table, B, T, max_rows, max_pages, num_pages, Hkv, D, codes,
//  scales, stream, ldk, ldv)
PyObject* cache_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_cache_append", args, n, 18);
        PyObject *K = a.next(), *V = a.next(), *start = a.next(), *pos = a.next(),
                 *table = a.next();
        const int B = a.integer(), T = a.integer(), max_rows = a.integer(),
                  max_pages = a.integer(), num_pages = a.integer(), Hkv = a.integer(),
                  D = a.integer();
        Cache cache{a.next(), a.next()};
        void* stream = a.stream();
        int ldk = 0, ldv = 0;
        const auto* k = rows(a, "K", K, T, Hkv, D, a.next(), ldk);
        const auto* v = rows(a, "V", V, T, Hkv, D, a.next(), ldv);
        cache.check(a, num_pages, Hkv, D);
        const auto* rs = array<int32_t>(a, "row_start", start, at::kInt, (long long)B + 1);
        const auto* ps = array<int32_t>(a, "pos", pos, at::kInt, B);
        const auto* pt = array<int32_t>(a, "page_table", table, at::kInt, product(B, max_pages));
        return call([&] {
            return lib.cache_append(k, v, rs, ps, pt, B, T, max_rows, max_pages, num_pages, Hkv,
                                    D, ldk, ldv, cache.c, cache.s, stream);
        });
    });
}

// (device, codes, scales, pages, n, num_pages, Hkv, D, K_out, V_out, stream)
PyObject* cache_dequant(PyObject*, PyObject* const* args, Py_ssize_t count) {
    return guarded([&] {
        Args a("rudder_cache_dequant", args, count, 11);
        Cache cache{a.next(), a.next()};
        PyObject* pages = a.next();
        const int n = a.integer(), num_pages = a.integer(), Hkv = a.integer(), D = a.integer();
        cache.check(a, num_pages, Hkv, D);
        const long long size = product(product(n, Hkv), product(RUDDER_CACHE_PAGE, D));
        const auto* p = array<int32_t>(a, "pages", pages, at::kInt, n);
        auto* k = array<float>(a, "K_out", a.next(), at::kFloat, size);
        auto* v = array<float>(a, "V_out", a.next(), at::kFloat, size);
        void* stream = a.stream();
        return call([&] {
            return lib.cache_dequant(cache.c, cache.s, p, n, num_pages, Hkv, D, k, v, stream);
        });
    });
}

// (device, Q, row_start, kv_len, page_table, codes, scales, B, T, max_rows, max_kv, max_pages,
//  num_pages, Hq, Hkv, D, sm, causal, workspace, O, stream, ldq, ldo)
PyObject* cache_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_cache_attention", args, n, 23);
        PyObject *Q = a.next(), *start = a.next(), *len = a.next(), *table = a.next();
        Cache cache{a.next(), a.next()};
        const int B = a.integer(), T = a.integer(), max_rows = a.integer(), max_kv = a.integer(),
                  max_pages = a.integer(), num_pages = a.integer(), Hq = a.integer(),
                  Hkv = a.integer(), D = a.integer();
        const float sm = a.real();
        const int causal = a.truth();
        size_t bytes = 0;
        void* ws = workspace(a, bytes);
        PyObject* O = a.next();
        void* stream = a.stream();
        int ldq = 0, ldo = 0;
        const auto* q = rows(a, "Q", Q, T, Hq, D, a.next(), ldq);
        auto* o = rows(a, "O", O, T, Hq, D, a.next(), ldo);
        cache.check(a, num_pages, Hkv, D);
        const auto* rs = array<int32_t>(a, "row_start", start, at::kInt, (long long)B + 1);
        const auto* kl = array<int32_t>(a, "kv_len", len, at::kInt, B);
        const auto* pt = array<int32_t>(a, "page_table", table, at::kInt, product(B, max_pages));
        return call([&] {
            return lib.cache_attention(q, rs, kl, pt, cache.c, cache.s, B, T, max_rows, max_kv,
                                       max_pages, num_pages, Hq, Hkv, D, ldq, ldo, sm, causal, ws,
                                       bytes, o, stream);
        });
    });
}

// (device, Q, K, V, row_start, kv_start, kv_len, B, T, Tkv, max_rows, max_kv, Hq, Hkv, D, sm,
//  workspace, O, stream, ldq, ldk, ldv, ldo)
PyObject* cross_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_cross_attention", args, n, 23);
        PyObject *Q = a.next(), *K = a.next(), *V = a.next(), *start = a.next(),
                 *kv_start = a.next(), *len = a.next();
        const int B = a.integer(), T = a.integer(), Tkv = a.integer(), max_rows = a.integer(),
                  max_kv = a.integer(), Hq = a.integer(), Hkv = a.integer(), D = a.integer();
        const float sm = a.real();
        size_t bytes = 0;
        void* ws = workspace(a, bytes);
        PyObject* O = a.next();
        void* stream = a.stream();
        int ldq = 0, ldk = 0, ldv = 0, ldo = 0;
        const auto* q = rows(a, "Q", Q, T, Hq, D, a.next(), ldq);
        const auto* k = rows(a, "K", K, Tkv, Hkv, D, a.next(), ldk);
        const auto* v = rows(a, "V", V, Tkv, Hkv, D, a.next(), ldv);
        auto* o = rows(a, "O", O, T, Hq, D, a.next(), ldo);
        const auto* rs = array<int32_t>(a, "row_start", start, at::kInt, (long long)B + 1);
        const auto* ks = array<int32_t>(a, "kv_start", kv_start, at::kInt, B);
        const auto* kl = array<int32_t>(a, "kv_len", len, at::kInt, B);
        return call([&] {
            return lib.cross_attention(q, k, v, rs, ks, kl, B, T, Tkv, max_rows, max_kv, Hq, Hkv,
                                       D, ldq, ldk, ldv, ldo, sm, ws, bytes, o, stream);
        });
    });
}

// (device, X, R, gamma, eps, M, K, H, Y, stream, ldx, ldr, ldh, ldy)
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_norm", args, n, 14);
        PyObject *X = a.next(), *R = a.next(), *gamma = a.next();
        const float eps = a.real();
        const int M = a.integer(), K = a.integer();
        PyObject *H = a.next(), *Y = a.next();
        void* stream = a.stream();
        int ldx = 0, ldr = 0, ldh = 0, ldy = 0;
        const auto* x = rows(a, "X", X, M, 1, K, a.next(), ldx);
        const auto* r = rows(a, "R", R, M, 1, K, a.next(), ldr);
        auto* h = rows(a, "H", H, M, 1, K, a.next(), ldh);
        auto* y = rows(a, "Y", Y, M, 1, K, a.next(), ldy);
        const auto* g = array<float>(a, "gamma", gamma, at::kFloat, K);
        return call([&] {
            return lib.norm(x, r, g, eps, M, K, ldx, ldr, ldh, ldy, h, y, stream);
        });
    });
}

// (device, X, R, stream_id, gamma, inv_smooth, act_scale, eps, M, K, S, abits, codes, H, Xq,
//  row_scale, stream, ldx, ldr, ldh)
PyObject* norm_quant(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_norm_quant", args, n, 20);
        PyObject *X = a.next(), *R = a.next(), *sid = a.next(), *gamma = a.next(),
                 *smooth = a.next(), *table = a.next();
        const float eps = a.real();
        const int M = a.integer(), K = a.integer(), S = a.integer(), abits = a.integer(),
                  codes = a.integer();
        PyObject *H = a.next(), *Xq = a.next(), *scale = a.next();
        void* stream = a.stream();
        int ldx = 0, ldr = 0, ldh = 0;
        const auto* x = rows(a, "X", X, M, 1, K, a.next(), ldx);
        const auto* r = rows(a, "R", R, M, 1, K, a.next(), ldr);
        auto* h = rows(a, "H", H, M, 1, K, a.next(), ldh);
        const auto* st = array<uint8_t>(a, "stream_id", sid, at::kByte, M);
        const auto* g = array<float>(a, "gamma", gamma, at::kFloat, K);
        const auto* is = array<float>(a, "inv_smooth", smooth, at::kFloat, K);
        const auto* d = array<float>(a, "act_scale", table, at::kFloat, S);
        auto* q = array<void>(a, "Xq", Xq, at::kByte,
                              (long long)lib.packed_act_bytes(M, K, abits, codes));
        auto* s = array<float>(a, "row_scale", scale, at::kFloat, M);
        return call([&] {
            return lib.norm_quant(x, r, st, g, is, d, eps, M, K, S, abits, codes, ldx, ldr, ldh, h,
                                  q, s, stream);
        });
    });
}

// (device, Xq, row_scale, M, K, abits, codes, out, stream)
PyObject* dequant_act(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_dequant_act", args, n, 9);
        PyObject *Xq = a.next(), *scale = a.next();
        const int M = a.integer(), K = a.integer(), abits = a.integer(), codes = a.integer();
        const auto* q = array<void>(a, "Xq", Xq, at::kByte,
                                    (long long)lib.packed_act_bytes(M, K, abits, codes));
        const auto* s = array<float>(a, "row_scale", scale, at::kFloat, M);
        auto* out = array<float>(a, "out", a.next(), at::kFloat, product(M, K));
        void* stream = a.stream();
        return call([&] { return lib.dequant_act(q, s, M, K, abits, codes, out, stream); });
    });
}

// (device, Q, K, row_start, pos, freq, magnitude, B, T, max_rows, Hq, Hkv, D, rotary_dim, layout,
//  Qo, Ko, stream, ldq, ldk, ldqo, ldko)
PyObject* rotary(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_rotary", args, n, 22);
        PyObject *Q = a.next(), *K = a.next(), *start = a.next(), *pos = a.next(),
                 *freq = a.next();
        const float magnitude = a.real();
        const int B = a.integer(), T = a.integer(), max_rows = a.integer(), Hq = a.integer(),
                  Hkv = a.integer(), D = a.integer(), part = a.integer(), layout = a.integer();
        PyObject *Qo = a.next(), *Ko = a.next();
        void* stream = a.stream();
        int ldq = 0, ldk = 0, ldqo = 0, ldko = 0;
        const auto* q = rows(a, "Q", Q, T, Hq, D, a.next(), ldq);
        const auto* k = rows(a, "K", K, T, Hkv, D, a.next(), ldk);
        auto* qo = rows(a, "Qo", Qo, T, Hq, D, a.next(), ldqo);
        auto* ko = rows(a, "Ko", Ko, T, Hkv, D, a.next(), ldko);
        const auto* rs = array<int32_t>(a, "row_start", start, at::kInt, (long long)B + 1);
        const auto* ps = array<int32_t>(a, "pos", pos, at::kInt, B);
        const auto* fr = array<double>(a, "freq", freq, at::kDouble, part / 2);
        return call([&] {
            return lib.rotary(q, k, rs, ps, fr, magnitude, B, T, max_rows, Hq, Hkv, D, part,
                              layout, ldq, ldk, ldqo, ldko, qo, ko, stream);
        });
    });
}

// (device, Q, K, V, row_start, B, T, max_rows, Hq, Hkv, D, sm, workspace, O, stream, ldq, ldk, ldv,
//  ldo)
PyObject* prompt_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a("rudder_prompt_attention", args, n, 19);
        PyObject *Q = a.next(), *K = a.next(), *V = a.next(), *start = a.next();
        const int B = a.integer(), T = a.integer(), max_rows = a.integer(), Hq = a.integer(),
                  Hkv = a.integer(), D = a.integer();
        const float sm = a.real();
        size_t bytes = 0;
        void* ws = workspace(a, bytes);
        PyObject* O = a.next();
        void* stream = a.stream();
        int ldq = 0, ldk = 0, ldv = 0, ldo = 0;
        const auto* q = rows(a, "Q", Q, T, Hq, D, a.next(), ldq);
        const auto* k = rows(a, "K", K, T, Hkv, D, a.next(), ldk);
        const auto* v = rows(a, "V", V, T, Hkv, D, a.next(), ldv);
        auto* o = rows(a, "O", O, T, Hq, D, a.next(), ldo);
        const auto* rs = array<int32_t>(a, "row_start", start, at::kInt, (long long)B + 1);
        return call([&] {
            return lib.prompt_attention(q, k, v, rs, B, T, max_rows, Hq, Hkv, D, ldq, ldk, ldv,
                                        ldo, sm, ws, bytes, o, stream);
        });
    });
}

// use(path): takes the entry points from the library loaded from there.
PyObject* use(PyObject*, PyObject* path) {
    const char* name = PyUnicode_AsUTF8(path);
    if (!name) return nullptr;
    void* h = dlopen(name, RTLD_NOW | RTLD_LOCAL);
    Library l = {};
    bool all = h != nullptr;
    auto find = [&](auto& f, const char* symbol) {
        if (all) f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, symbol));
        all = all && f;
    };
    find(l.quantize_weights_grouped, "rudder_quantize_weights_grouped");
    find(l.matvec_w4, "rudder_matvec_w4");
    find(l.grouped_weight_bytes, "rudder_grouped_weight_bytes");
    find(l.grouped_scale_count, "rudder_grouped_scale_count");
    find(l.cache_append, "rudder_cache_append");
    find(l.cache_dequant, "rudder_cache_dequant");
    find(l.cache_attention, "rudder_cache_attention");
    find(l.cross_attention, "rudder_cross_attention");
    find(l.packed_act_bytes, "rudder_packed_act_bytes");
    find(l.norm, "rudder_norm");
    find(l.norm_quant, "rudder_norm_quant");
    find(l.dequant_act, "rudder_dequant_act");
    find(l.rotary, "rudder_rotary");
    find(l.prompt_attention, "rudder_prompt_attention");
    if (!all) return PyErr_Format(PyExc_ImportError, "%s: %s", name, dlerror());
    lib = l;
    Py_RETURN_NONE;
}

#define RUDDER_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), \
                          METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"use", use, METH_O, nullptr},
    RUDDER_METHOD(quantize_weights_grouped),
    RUDDER_METHOD(matvec_w4),
    RUDDER_METHOD(cache_append),
    RUDDER_METHOD(cache_dequant),
    RUDDER_METHOD(cache_attention),
    RUDDER_METHOD(cross_attention),
    RUDDER_METHOD(norm),
    RUDDER_METHOD(norm_quant),
    RUDDER_METHOD(dequant_act),
    RUDDER_METHOD(rotary),
    RUDDER_METHOD(prompt_attention),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rudder_bind",
                      "Argument checks and calls of the operators around and between the linears.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rudder_bind() { return PyModule_Create(&module); }
