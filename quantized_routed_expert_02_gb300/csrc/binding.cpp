// Python entry points of the attention half (module _binding): argument checks
// on the tensors themselves, then the C ABI's own.
//
// These calls take up to 13 tensors each, and a single token's kernel is done in
// 3 to 6 us: in Python the checks and the conversion of the arguments take
// longer than that (7 us of a call's 10), here under a microsecond.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAStream.h>

#include <cstring>
#include <initializer_list>
#include <string>

#include "moeq4k.h"

namespace {

PyObject *moe_error = nullptr;  // the exception of a refused call: (code, where)

// A Python exception is set: unwinds to the entry point.
struct Raised {};

[[noreturn]] void refuse(PyObject *type, const std::string &text) {
    PyErr_SetString(type, text.c_str());
    throw Raised();
}

std::string dtype_name(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kDouble: return "torch.float64";
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kChar: return "torch.int8";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

std::string shape_text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + ": not a tensor");
    return THPVariable_Unpack(o);
}

// The sizes of a tensor of n dimensions.
at::IntArrayRef sizes(const at::Tensor &t, size_t n, const char *name) {
    if (t.sizes().size() != n)
        refuse(PyExc_ValueError, std::string(name) + ": shape " + shape_text(t.sizes()) + " has not " +
                                    std::to_string(n) + " dimensions");
    return t.sizes();
}

// The device of a call's first tensor, where all the others have to be too.
struct Place {
    c10::Device device;
    bool current;  // the CUDA device that a call is launched on

    explicit Place(const at::Tensor &first)
        : device(first.device()),
          current(device.is_cuda() && device.index() == c10::cuda::current_device()) {}
    void check(const at::Tensor &t, const char *name) const {
        if (t.device() != device)
            refuse(PyExc_ValueError, std::string(name) + ": on " + t.device().str() + ", not " + device.str());
    }
    // The pointer of a contiguous tensor of this shape and type.
    template <typename P = void>
    P *pointer(const at::Tensor &t, at::IntArrayRef shape, at::ScalarType type, const char *name) const;
    template <typename P = void>
    P *pointer(PyObject *o, at::IntArrayRef shape, at::ScalarType type, const char *name) const {
        return pointer<P>(tensor(o, name), shape, type, name);
    }
    template <typename P = void>
    P *optional(PyObject *o, at::IntArrayRef shape, at::ScalarType type, const char *name) const {
        return o == Py_None ? nullptr : pointer<P>(o, shape, type, name);
    }
    // A workspace's size is that of its bytes in a row: an expanded view has more elements than bytes.
    void *workspace(const at::Tensor &t) const {
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "ws: not contiguous");
        check(t, "ws");
        return t.data_ptr();
    }
};

template <typename P>
P *Place::pointer(const at::Tensor &t, at::IntArrayRef shape, at::ScalarType type, const char *name) const {
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, std::string(name) + ": " + dtype_name(t.scalar_type()) + ", not " + dtype_name(type));
    if (t.sizes() != shape)
        refuse(PyExc_ValueError,
              std::string(name) + ": shape " + shape_text(t.sizes()) + ", not " + shape_text(shape));
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + ": not contiguous");
    check(t, name);
    return static_cast<P *>(t.data_ptr());
}

moe_dtype dtype_of(const at::Tensor &t, const char *name) {
    switch (t.scalar_type()) {
        case at::kFloat: return MOE_F32;
        case at::kHalf: return MOE_F16;
        case at::kBFloat16: return MOE_BF16;
        default:
            refuse(PyExc_TypeError, std::string(name) + ": " + dtype_name(t.scalar_type()) +
                                       " is not one of float32, float16, bfloat16");
    }
}

int as_int(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    if (v != int(v)) refuse(PyExc_OverflowError, "not a 32-bit integer: " + std::to_string(v));
    return int(v);
}

int extent(int64_t v, const char *name) {
    if (v != int(v)) refuse(PyExc_ValueError, std::string(name) + ": " + std::to_string(v) + " is past 32 bits");
    return int(v);
}

float as_float(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return float(v);
}

// None: the current stream; a torch.cuda.Stream; or a handle.  Tensors that the
// current device does not hold: their call is checked only (run() refuses it then).
void *as_stream(PyObject *o, const Place &place) {
    if (!place.current) return MOE_CHECK_ONLY;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *h = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (h == nullptr) throw Raised();
    void *s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (s == nullptr && PyErr_Occurred()) throw Raised();
    if (s == MOE_CHECK_ONLY) refuse(PyExc_ValueError, "stream: not a stream's handle: -1");
    return s;
}

// The arguments in the order of `names`; those from `required` on may be left
// out (the value given here, borrowed).
template <size_t N>
struct Args {
    PyObject *v[N];

    Args(const char *call, const char *const (&names)[N], size_t required, PyObject *const *args, Py_ssize_t n,
         PyObject *kwnames) {
        for (PyObject *&a : v) a = nullptr;
        if (n > Py_ssize_t(N))
            refuse(PyExc_TypeError, std::string(call) + "() takes " + std::to_string(N) + " arguments, " +
                                       std::to_string(n) + " given");
        for (Py_ssize_t i = 0; i < n; ++i) v[i] = args[i];
        const Py_ssize_t nk = kwnames == nullptr ? 0 : PyTuple_GET_SIZE(kwnames);
        for (Py_ssize_t k = 0; k < nk; ++k) {
            const char *key = PyUnicode_AsUTF8(PyTuple_GET_ITEM(kwnames, k));
            if (key == nullptr) throw Raised();
            size_t i = 0;
            while (i < N && std::strcmp(names[i], key) != 0) ++i;
            if (i == N)
                refuse(PyExc_TypeError, std::string(call) + "() got an unexpected keyword argument '" + key + "'");
            if (v[i] != nullptr)
                refuse(PyExc_TypeError, std::string(call) + "() got multiple values for argument '" + key + "'");
            v[i] = args[n + k];
        }
        for (size_t i = 0; i < N; ++i) {
            if (v[i] != nullptr) continue;
            if (i < required)
                refuse(PyExc_TypeError, std::string(call) + "() missing argument '" + names[i] + "'");
            v[i] = Py_None;
        }
    }
    PyObject *operator[](size_t i) const { return v[i]; }
};

// Runs `call` without the interpreter's lock (a launch may wait for room in the
// queue) and raises what it refuses; then, what the library cannot see, tensors that
// are not where it would be launched.
template <typename F>
void run(const char *where, const Place &place, F call) {
    moe_status code;
    Py_BEGIN_ALLOW_THREADS;
    code = call();
    Py_END_ALLOW_THREADS;
    if (code == MOE_OK && place.current) return;
    if (code == MOE_OK)
        refuse(PyExc_ValueError, std::string(where) + ": tensors on " + place.device.str() +
                                     ", which is not the current CUDA device");
    PyObject *e = PyObject_CallFunction(moe_error, "is", int(code), where);
    if (e != nullptr) {
        PyErr_SetObject(moe_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

template <typename F>
PyObject *entry(F body) {
    try {
        body();
        Py_RETURN_NONE;
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *add_rmsnorm(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) {
    return entry([&] {
        static const char *const names[] = {"x", "residual", "gamma", "eps", "sum_out", "y", "q8k", "stream"};
        const Args<8> a("moe_add_rmsnorm", names, 4, args, n, kwnames);
        const at::Tensor &x = tensor(a[0], "x");
        const Place at_x(x);
        const at::IntArrayRef rows = sizes(x, 2, "x");
        const int T = extent(rows[0], "x"), H = extent(rows[1], "x");
        int8_t *q = nullptr;
        float *d = nullptr;
        int32_t *sums = nullptr;
        if (a[6] != Py_None) {
            if (!(PyTuple_Check(a[6]) || PyList_Check(a[6])) || PySequence_Fast_GET_SIZE(a[6]) != 3)
                refuse(PyExc_TypeError, "q8k: not a tuple (q, d, sums)");
            q = at_x.pointer<int8_t>(PySequence_Fast_GET_ITEM(a[6], 0), rows, at::kChar, "q");
            d = at_x.pointer<float>(PySequence_Fast_GET_ITEM(a[6], 1), {T, H / 256}, at::kFloat, "d");
            sums = at_x.pointer<int32_t>(PySequence_Fast_GET_ITEM(a[6], 2), {T, H / 32}, at::kInt, "sums");
        }
        const moe_dtype xt = dtype_of(x, "x");
        const void *xp = at_x.pointer(x, rows, x.scalar_type(), "x");
        const float *residual = at_x.optional<float>(a[1], rows, at::kFloat, "residual");
        const float *gamma = at_x.pointer<float>(a[2], {H}, at::kFloat, "gamma");
        const float eps = as_float(a[3]);
        float *sum_out = at_x.optional<float>(a[4], rows, at::kFloat, "sum_out");
        void *y = nullptr;
        moe_dtype yt = MOE_F32;
        if (a[5] != Py_None) {
            const at::Tensor &t = tensor(a[5], "y");
            yt = dtype_of(t, "y");
            y = at_x.pointer(t, rows, t.scalar_type(), "y");
        }
        void *s = as_stream(a[7], at_x);
        run("moe_add_rmsnorm", at_x, [&] {
            return moe_add_rmsnorm(xp, xt, residual, gamma, eps, T, H, sum_out, y, yt, q, d, sums, s);
        });
    });
}

// The paged cache and the batch of the next two.
struct Cache : Place {
    void *k, *v;
    const int32_t *table, *offs, *lens;
    int B, max_pages, pages, page, Hkv, D;
    at::ScalarType type;
    moe_dtype dtype;

    Cache(PyObject *kp, PyObject *vp, PyObject *table_, PyObject *offs_, PyObject *lens_)
        : Place(tensor(kp, "k_pages")) {
        const at::Tensor &kt = tensor(kp, "k_pages"), &tt = tensor(table_, "page_table");
        const at::IntArrayRef c = sizes(kt, 4, "k_pages"), t = sizes(tt, 2, "page_table");
        pages = extent(c[0], "k_pages"), Hkv = extent(c[1], "k_pages");
        page = extent(c[2], "k_pages"), D = extent(c[3], "k_pages");
        B = extent(t[0], "page_table"), max_pages = extent(t[1], "page_table");
        type = kt.scalar_type();
        dtype = dtype_of(kt, "k_pages");
        k = pointer(kt, c, type, "k_pages");
        v = pointer(vp, c, type, "v_pages");
        table = pointer<int32_t>(tt, t, at::kInt, "page_table");
        offs = pointer<int32_t>(offs_, {B + 1}, at::kInt, "q_offs");
        lens = pointer<int32_t>(lens_, {B}, at::kInt, "kv_lens");
    }
};

PyObject *rope_append(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) {
    return entry([&] {
        static const char *const names[] = {"qkv",    "pos",     "inv_freq", "q_out", "k_pages",  "v_pages",
                                            "page_table", "q_offs", "kv_lens", "ws",  "axis",     "q_norm_w",
                                            "k_norm_w", "eps",   "interleaved", "stream"};
        const Args<16> a("moe_rope_append", names, 10, args, n, kwnames);
        const Cache c(a[4], a[5], a[6], a[7], a[8]);
        const at::Tensor &out = tensor(a[3], "q_out"), &pos = tensor(a[1], "pos"), &freq = tensor(a[2], "inv_freq");
        const at::IntArrayRef o = sizes(out, 3, "q_out");
        const int N = extent(o[0], "q_out"), Hq = extent(o[1], "q_out");
        const int axes = extent(sizes(pos, 2, "pos")[0], "pos");
        const int half = extent(sizes(freq, 1, "inv_freq")[0], "inv_freq");
        const void *qkv = c.pointer(a[0], {N, int64_t(Hq + 2 * int64_t(c.Hkv)) * c.D}, c.type, "qkv");
        const int32_t *at_pos = c.pointer<int32_t>(pos, {axes, N}, at::kInt, "pos");
        const double *f = c.pointer<double>(freq, {half}, at::kDouble, "inv_freq");
        const int32_t *axis = c.optional<int32_t>(a[10], {half}, at::kInt, "axis");
        const float *qw = c.optional<float>(a[11], {c.D}, at::kFloat, "q_norm_w");
        const float *kw = c.optional<float>(a[12], {c.D}, at::kFloat, "k_norm_w");
        const float eps = a[13] == Py_None ? 1e-6f : as_float(a[13]);
        const int turned = a[14] == Py_None ? 0 : PyObject_IsTrue(a[14]);
        if (turned < 0) throw Raised();
        void *q_out = c.pointer(out, {N, Hq, c.D}, c.type, "q_out");
        const at::Tensor &ws = tensor(a[9], "ws");
        void *w = c.workspace(ws), *s = as_stream(a[15], c);
        run("moe_rope_append", c, [&] {
            return moe_rope_append(qkv, at_pos, f, axis, axes, 2 * half, turned, qw, kw, eps, q_out, c.k, c.v,
                                   c.table, c.offs, c.lens, N, c.B, c.max_pages, c.pages, c.page, Hq, c.Hkv, c.D,
                                   c.dtype, w, ws.nbytes(), s);
        });
    });
}

PyObject *attention_paged(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) {
    return entry([&] {
        static const char *const names[] = {"q",     "k_pages", "v_pages", "page_table", "q_offs", "kv_lens", "max_new",
                                            "scale", "out",     "ws",      "lse",        "window", "softcap", "stream"};
        const Args<14> a("moe_attention_paged", names, 10, args, n, kwnames);
        const Cache c(a[1], a[2], a[3], a[4], a[5]);
        const at::Tensor &qt = tensor(a[0], "q");
        const at::IntArrayRef r = sizes(qt, 3, "q");
        const int N = extent(r[0], "q"), Hq = extent(r[1], "q");
        const void *q = c.pointer(qt, {N, Hq, c.D}, c.type, "q");
        const int most = as_int(a[6]), window = a[11] == Py_None ? 0 : as_int(a[11]);
        const float scale = as_float(a[7]), softcap = a[12] == Py_None ? 0.f : as_float(a[12]);
        void *out = c.pointer(a[8], {N, Hq, c.D}, c.type, "out");
        float *lse = c.optional<float>(a[10], {N, Hq}, at::kFloat, "lse");
        const at::Tensor &ws = tensor(a[9], "ws");
        void *w = c.workspace(ws), *s = as_stream(a[13], c);
        run("moe_attention_paged", c, [&] {
            return moe_attention_paged(q, c.k, c.v, c.table, c.offs, c.lens, N, c.B, most, c.max_pages, c.pages,
                                       c.page, Hq, c.Hkv, c.D, c.dtype, scale, softcap, window, out, lse, w,
                                       ws.nbytes(), s);
        });
    });
}

PyObject *set_error(PyObject *, PyObject *type) {
    Py_XSETREF(moe_error, Py_NewRef(type));
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS

PyMethodDef methods[] = {
    {"moe_add_rmsnorm", FAST(add_rmsnorm),
     "moe_add_rmsnorm(x, residual, gamma, eps, sum_out=None, y=None, q8k=None, stream=None)\n--\n\n"
     "s = x + residual (None: s = x), y = RMSNorm(s) * gamma.  ``sum_out`` receives s, ``y`` the\n"
     "normed rows (fp32, fp16 or bf16), ``q8k`` = (q, d, sums) their Q8_K blocks."},
    {"moe_rope_append", FAST(rope_append),
     "moe_rope_append(qkv, pos, inv_freq, q_out, k_pages, v_pages, page_table, q_offs, kv_lens, ws,\n"
     "                axis=None, q_norm_w=None, k_norm_w=None, eps=1e-6, interleaved=False,\n"
     "                stream=None)\n--\n\n"
     "Rows ``qkv`` [N, (Hq + 2 Hkv) D] -> normed and rotated queries ``q_out`` [N, Hq, D], keys\n"
     "(normed, rotated) and values into the cache.  ``pos`` int32 [axes, N], ``inv_freq`` float64\n"
     "[rot / 2] radians per position, ``axis`` int32 [rot / 2]: the axis of each pair."},
    {"moe_attention_paged", FAST(attention_paged),
     "moe_attention_paged(q, k_pages, v_pages, page_table, q_offs, kv_lens, max_new, scale, out, ws,\n"
     "                    lse=None, window=0, softcap=0.0, stream=None)\n--\n\n"
     "Attention of the new rows ``q`` [N, Hq, D] over each sequence's cached tokens -> ``out``\n"
     "[N, Hq, D], ``lse`` [N, Hq] (optional).  ``max_new``: the most new tokens of a sequence."},
    {"set_error", set_error, METH_O, "The exception type of refused calls."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Entry points of the attention half.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
