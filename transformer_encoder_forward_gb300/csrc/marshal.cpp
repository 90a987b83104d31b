// Argument marshalling of the binding's calls whose device time is a few
// microseconds: reads the tensors' addresses, sizes and types through
// PyTorch's C++ interface (a read of each through Python costs as much as a
// launch), checks them and calls the C ABI, without the interpreter's lock (a
// launch may wait for room in its stream, behind a callback that needs the
// lock).  Holds no arithmetic.  Every function returns the te_status; the Python
// side raises for it.
// The C ABI's functions are the ones of the library that the binding has
// loaded: it hands over their addresses once (bind), so the module is linked
// against no second copy.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <string>
#include <vector>

#include "tefwd.h"

namespace {

struct {
    decltype(&te_quant_rows) quant_rows;
    decltype(&te_rownorm_quant) rownorm_quant;
    decltype(&te_i8_linear) i8_linear;
    decltype(&te_i8_gated_linear) i8_gated_linear;
    decltype(&te_qk_rope_axes) qk_rope_axes;
    decltype(&te_attn_sink_fwd) attn_sink_fwd;
    decltype(&te_attn_relbias_fwd) attn_relbias_fwd;
} abi;

struct PyError {};   // a Python exception is set

[[noreturn]] void raise(PyObject *type, const std::string &msg) {
    PyErr_SetString(type, msg.c_str());
    throw PyError();
}

// The sizes and address of a tensor argument.
struct Arg {
    void *ptr;
    int64_t rows, cols, ld;
    int dtype;   // TE_F32 / TE_BF16, or -1
};

enum Types { F32 = 1, BF16 = 2, I8 = 4, I32 = 8 };

// A matrix [rows, cols] (dims == 2) or vector [cols] (dims == 1) on the current
// device with a contiguous last axis; -1: any size.
Arg want(const char *what, PyObject *o, int types, int dims, int64_t rows, int64_t cols) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(what) + ": not a tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    const at::ScalarType st = t.scalar_type();
    const int have = st == at::kFloat ? F32 : st == at::kBFloat16 ? BF16 : st == at::kChar ? I8 : st == at::kInt ? I32 : 0;
    if (!(have & types)) raise(PyExc_TypeError, std::string(what) + ": dtype " + c10::toString(st));
    if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
        raise(PyExc_ValueError, std::string(what) + ": a tensor on the current CUDA device, not on " + t.device().str());
    if (t.dim() != dims || (dims == 2 && rows >= 0 && t.size(0) != rows) || (cols >= 0 && t.size(-1) != cols)) {
        std::string s = std::string(what) + ": shape [";
        for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
        s += "], not [";
        if (dims == 2) s += rows >= 0 ? std::to_string(rows) + ", " : "any, ";
        raise(PyExc_ValueError, s + (cols >= 0 ? std::to_string(cols) : "any") + "]");
    }
    if (t.size(-1) > 1 && t.stride(-1) != 1)
        raise(PyExc_ValueError, std::string(what) + ": its last axis must be contiguous");
    Arg a;
    a.ptr = t.data_ptr();
    a.rows = dims == 2 ? t.size(0) : 1;
    a.cols = t.size(-1);
    a.ld = dims == 2 ? t.stride(0) : a.cols;
    if (a.rows == 1) a.ld = (a.cols + 15) / 16 * 16;    // a single row's stride says nothing
    if (a.rows > 2147483647 || a.cols > 2147483647) raise(PyExc_ValueError, std::string(what) + ": too large");
    a.dtype = have == F32 ? TE_F32 : have == BF16 ? TE_BF16 : -1;
    return a;
}

// A leading dimension that the caller gives beside the tensor it belongs to.
int64_t leading(const char *what, const Arg &t, int64_t ld) {
    if (t.rows > 1 && ld != t.ld)
        raise(PyExc_ValueError, std::string(what) + ": leading dimension " + std::to_string(ld) + ", the tensor's is " +
                                    std::to_string(t.ld));
    return ld;
}

void *opt(const char *what, PyObject *o, int types, int64_t cols) {
    return o == Py_None ? nullptr : want(what, o, types, 1, 1, cols).ptr;
}

// A workspace: any contiguous tensor on the current device, or None.
void *scratch(const char *what, PyObject *o, size_t &bytes) {
    bytes = 0;
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(what) + ": the workspace must be a tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != c10::cuda::current_device() || !t.is_contiguous())
        raise(PyExc_ValueError, std::string(what) + ": the workspace must be a contiguous tensor on the current CUDA device");
    bytes = (size_t)t.numel() * t.element_size();
    return t.data_ptr();
}

te_stream stream_of(PyObject *o) {
    if (o == Py_None) return reinterpret_cast<te_stream>(c10::cuda::getCurrentCUDAStream().stream());
    PyObject *v = PyObject_GetAttrString(o, "cuda_stream");
    if (!v) throw PyError();
    void *s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!s && PyErr_Occurred()) throw PyError();
    return static_cast<te_stream>(s);
}

long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyError();
    return v;
}
int32_t int32_of(PyObject *o) {
    const long long v = integer(o);
    if (v < -2147483648ll || v > 2147483647ll) raise(PyExc_OverflowError, "an int32 argument out of range");
    return (int32_t)v;
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyError();
    return (float)v;
}

// A ctypes structure of the C ABI.
template <typename T>
T structure(const char *what, PyObject *o) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw PyError();
    T v;
    const bool ok = b.len == (Py_ssize_t)sizeof(T);
    if (ok) memcpy(&v, b.buf, sizeof(T));
    PyBuffer_Release(&b);
    if (!ok) raise(PyExc_TypeError, std::string(what) + ": not the structure expected");
    return v;
}

void count(Py_ssize_t have, Py_ssize_t need) {
    if (have != need) raise(PyExc_TypeError, "wrong number of arguments");
}
// The same for a call of the C ABI.
void call_args(Py_ssize_t have, Py_ssize_t need) {
    if (!abi.quant_rows) raise(PyExc_RuntimeError, "the library's functions have not been bound");
    count(have, need);
}

// Runs f (a te_status), turning C++ exceptions into Python ones.
template <typename F>
PyObject *guarded(F f) {
    try {
        return PyLong_FromLong((long)f());
    } catch (const PyError &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// Runs f, a call of the C ABI on arguments that were read before, while other
// Python threads may run.
template <typename F>
te_status unlocked(F f) {
    PyThreadState *state = PyEval_SaveThread();
    const te_status st = f();
    PyEval_RestoreThread(state);
    return st;
}

// quant_rows(x, q, scale, stream)
PyObject *quant_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        call_args(n, 4);
        const Arg x = want("quant_rows: x", a[0], F32 | BF16, 2, -1, -1);
        const Arg q = want("quant_rows: q", a[1], I8, 2, x.rows, x.cols);
        const Arg s = want("quant_rows: scale", a[2], F32, 1, 1, x.rows);
        te_stream stream = stream_of(a[3]);
        return unlocked([&] {
            return abi.quant_rows(x.ptr, x.dtype, x.ld, static_cast<int8_t *>(q.ptr), q.ld, static_cast<float *>(s.ptr),
                                  (int32_t)x.rows, (int32_t)x.cols, stream);
        });
    });
}

// rownorm_quant(x, w, b, kind, eps, q, scale, pre, mod_scale, stream)
PyObject *rownorm_quant(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        call_args(n, 10);
        const Arg x = want("rownorm_quant: x", a[0], F32 | BF16, 2, -1, -1);
        const void *w = want("rownorm_quant: w", a[1], F32, 1, 1, x.cols).ptr;
        const void *b = opt("rownorm_quant: b", a[2], F32, x.cols);
        const Arg q = want("rownorm_quant: q", a[5], I8, 2, x.rows, x.cols);
        const Arg s = want("rownorm_quant: scale", a[6], F32, 1, 1, x.rows);
        const void *m = opt("rownorm_quant: mod_scale", a[8], F32, x.cols);
        const int32_t kind = int32_of(a[3]);
        const float eps = real(a[4]), pre = real(a[7]);
        te_stream stream = stream_of(a[9]);
        return unlocked([&] {
            return abi.rownorm_quant(x.ptr, x.dtype, x.ld, static_cast<const float *>(w), static_cast<const float *>(b),
                                     static_cast<const float *>(m), kind, eps, pre, static_cast<int8_t *>(q.ptr), q.ld,
                                     static_cast<float *>(s.ptr), (int32_t)x.rows, (int32_t)x.cols, stream);
        });
    });
}

// A key of an item's dict, or nullptr.
PyObject *key(PyObject *item, PyObject *name) {
    PyObject *v = PyDict_GetItemWithError(item, name);   // borrowed
    if (!v && PyErr_Occurred()) throw PyError();
    return v;
}
PyObject *K_W, *K_Y, *K_LDY, *K_RESIDUAL, *K_LDR, *K_EPILOGUE;

// i8_linear(xq, x_scale, items, workspace, stream)
PyObject *i8_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        call_args(n, 5);
        const Arg x = want("i8_linear: xq", a[0], I8, 2, -1, -1);
        const Arg s = want("i8_linear: x_scale", a[1], F32, 1, 1, x.rows);
        PyObject *seq = PySequence_Fast(a[2], "i8_linear: items must be a sequence");
        if (!seq) throw PyError();
        te_q8_item items[8];
        const Py_ssize_t z = PySequence_Fast_GET_SIZE(seq);
        try {
            if (z > 8) raise(PyExc_ValueError, "i8_linear: too many items");
            for (Py_ssize_t i = 0; i < z; ++i) {
                PyObject *it = PySequence_Fast_GET_ITEM(seq, i);
                if (!PyDict_Check(it)) raise(PyExc_TypeError, "i8_linear: an item is a dict");
                PyObject *w = key(it, K_W), *y = key(it, K_Y), *ldy = key(it, K_LDY), *r = key(it, K_RESIDUAL),
                         *e = key(it, K_EPILOGUE);
                if (!w || !y || !ldy) raise(PyExc_KeyError, "i8_linear: an item needs w, y and ldy");
                te_q8_item &d = items[i];
                d.w = structure<te_q8w>("i8_linear: w", w);
                const Arg ya = want("i8_linear: y", y, F32 | BF16, 2, x.rows, d.w.n);
                d.y = ya.ptr;
                d.ldy = leading("i8_linear: y", ya, integer(ldy));
                d.y_dtype = ya.dtype;
                d.epilogue = e ? int32_of(e) : TE_EPI_NONE;
                d.residual = nullptr;
                d.ldr = 0;
                if (r && r != Py_None) {
                    PyObject *ldr = key(it, K_LDR);
                    if (!ldr) raise(PyExc_KeyError, "i8_linear: a residual needs ldr");
                    const Arg ra = want("i8_linear: residual", r, F32, 2, x.rows, -1);
                    if (ra.cols < d.w.n) raise(PyExc_ValueError, "i8_linear: residual: fewer columns than features");
                    d.residual = static_cast<const float *>(ra.ptr);
                    d.ldr = leading("i8_linear: residual", ra, integer(ldr));
                }
            }
        } catch (...) {
            Py_DECREF(seq);
            throw;
        }
        Py_DECREF(seq);
        size_t nb;
        void *ws = scratch("i8_linear", a[3], nb);
        te_stream stream = stream_of(a[4]);
        return unlocked([&] {
            return abi.i8_linear(static_cast<const int8_t *>(x.ptr), x.ld, static_cast<const float *>(s.ptr),
                                 (int32_t)x.rows, (int32_t)x.cols, items, (int32_t)z, ws, nb, stream);
        });
    });
}

// i8_gated_linear(xq, x_scale, wg, wu, act, out, workspace, stream)
PyObject *i8_gated_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        call_args(n, 8);
        const Arg x = want("i8_gated_linear: xq", a[0], I8, 2, -1, -1);
        const Arg s = want("i8_gated_linear: x_scale", a[1], F32, 1, 1, x.rows);
        const te_q8w wg = structure<te_q8w>("i8_gated_linear: wg", a[2]);
        const te_q8w wu = structure<te_q8w>("i8_gated_linear: wu", a[3]);
        const Arg o = want("i8_gated_linear: out", a[5], BF16, 2, x.rows, wg.n);
        size_t nb;
        void *ws = scratch("i8_gated_linear", a[6], nb);
        const int32_t act = int32_of(a[4]);
        te_stream stream = stream_of(a[7]);
        return unlocked([&] {
            return abi.i8_gated_linear(static_cast<const int8_t *>(x.ptr), x.ld, static_cast<const float *>(s.ptr),
                                       (int32_t)x.rows, (int32_t)x.cols, &wg, &wu, act, o.ptr, o.ld, ws, nb, stream);
        });
    });
}

// qk_rope_axes(src, ld_src, dst, ld_dst, q_off, k_off, nq, nkv, hd, qn, kn, eps, plan, pos, q_mul, rows, stream)
PyObject *qk_rope_axes(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        call_args(n, 17);
        const int32_t rows = int32_of(a[15]), hd = int32_of(a[8]);
        const Arg src = want("qk_rope_axes: src", a[0], F32 | BF16, 2, rows, -1);
        const Arg dst = want("qk_rope_axes: dst", a[2], src.dtype == TE_F32 ? F32 : BF16, 2, rows, -1);
        const te_rope_axes plan = structure<te_rope_axes>("qk_rope_axes: plan", a[12]);
        const Arg pos = want("qk_rope_axes: pos", a[13], I32, 2, rows, plan.axes);
        const int64_t lds = leading("qk_rope_axes: src", src, integer(a[1]));
        const int64_t ldd = leading("qk_rope_axes: dst", dst, integer(a[3]));
        const int32_t q_off = int32_of(a[4]), k_off = int32_of(a[5]), nq = int32_of(a[6]), nkv = int32_of(a[7]);
        const int64_t end = std::max(nq ? q_off + (int64_t)nq * hd : 0, nkv ? k_off + (int64_t)nkv * hd : 0);
        if (end > src.cols || end > dst.cols)
            raise(PyExc_ValueError, "qk_rope_axes: the heads end at column " + std::to_string(end) + " of " +
                                        std::to_string(std::min(src.cols, dst.cols)));
        const float *qn = static_cast<const float *>(opt("qk_rope_axes: qn", a[9], F32, hd));
        const float *kn = static_cast<const float *>(opt("qk_rope_axes: kn", a[10], F32, hd));
        const float eps = real(a[11]), q_mul = real(a[14]);
        te_stream stream = stream_of(a[16]);
        return unlocked([&] {
            return abi.qk_rope_axes(src.ptr, lds, dst.ptr, ldd, src.dtype, q_off, k_off, nq, nkv, hd, qn, kn, eps, &plan,
                                    static_cast<const int32_t *>(pos.ptr), pos.ld, q_mul, rows, stream);
        });
    });
}

// The packed batch of an attention call: the panel, the output, and the
// sequences' offsets on the host (a contiguous int32 buffer, released at the end).
struct Batch {
    Arg qkv, out, cu_dev;
    Py_buffer cu;
    const int32_t *offsets;
    int32_t nseq;
    Batch(const std::string &name, PyObject *panel, PyObject *host, PyObject *dev, PyObject *o) {
        if (PyObject_GetBuffer(host, &cu, PyBUF_CONTIG_RO | PyBUF_FORMAT) != 0) throw PyError();
        try {
            const std::string f = cu.format ? cu.format : "B";
            if (cu.ndim != 1 || cu.itemsize != 4 || (f != "i" && f != "=i" && f != "<i" && f != "l" && f != "<l"))
                raise(PyExc_TypeError, name + ": cu_host: not a vector of int32");
            if (cu.shape[0] < 2 || cu.shape[0] > 2147483647) raise(PyExc_ValueError, name + ": cu_host: no sequence");
            offsets = static_cast<const int32_t *>(cu.buf);
            nseq = (int32_t)(cu.shape[0] - 1);
            cu_dev = want((name + ": cu_dev").c_str(), dev, I32, 1, 1, nseq + 1);
            qkv = want((name + ": qkv").c_str(), panel, BF16, 2, -1, -1);
            out = want((name + ": out").c_str(), o, BF16, 2, -1, -1);
            if (qkv.rows < offsets[nseq] || out.rows < offsets[nseq])
                raise(PyExc_ValueError, name + ": the sequences end at row " + std::to_string(offsets[nseq]) + " of " +
                                            std::to_string(std::min(qkv.rows, out.rows)));
        } catch (...) {
            PyBuffer_Release(&cu);
            throw;
        }
    }
    Batch(const Batch &) = delete;
    ~Batch() { PyBuffer_Release(&cu); }
};

void inside(const char *what, int64_t end, const Arg &t) {
    if (end > t.cols)
        raise(PyExc_ValueError, std::string(what) + ": the heads end at column " + std::to_string(end) + " of " + std::to_string(t.cols));
}

// attn_sink_fwd(qkv, ld, q_off, k_off, v_off, cu_host, cu_dev, nq, nkv, hd, left, right, sinks, scale, out, ldo, stream)
// attn_relbias_fwd(..., scale, plan, table, out, ldo, stream)
template <bool BIAS>
PyObject *attn_span(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        call_args(n, BIAS ? 19 : 17);
        const char *name = BIAS ? "attn_relbias_fwd" : "attn_sink_fwd";
        PyObject *const *t = a + (BIAS ? 16 : 14);   // out, ldo, stream
        const int32_t q_off = int32_of(a[2]), k_off = int32_of(a[3]), v_off = int32_of(a[4]);
        const int32_t nq = int32_of(a[7]), nkv = int32_of(a[8]), hd = int32_of(a[9]);
        const int32_t left = int32_of(a[10]), right = int32_of(a[11]), sinks = int32_of(a[12]);
        const float scale = real(a[13]);
        const int64_t ld = integer(a[1]), ldo = integer(t[1]);
        te_stream stream = stream_of(t[2]);
        te_relpos plan;
        Arg table;
        if (BIAS) {
            plan = structure<te_relpos>("attn_relbias_fwd: plan", a[14]);
            table = want("attn_relbias_fwd: table", a[15], F32, 2, plan.buckets, -1);
            if (table.cols < nq) raise(PyExc_ValueError, "attn_relbias_fwd: table: fewer columns than heads");
        }
        const Batch b(name, a[0], a[5], a[6], t[0]);
        leading(name, b.qkv, ld);
        leading(name, b.out, ldo);
        inside(name, std::max(q_off + (int64_t)nq * hd, std::max(k_off, v_off) + (int64_t)nkv * hd), b.qkv);
        inside(name, (int64_t)nq * hd, b.out);
        return unlocked([&] {
            if (BIAS)
                return abi.attn_relbias_fwd(b.qkv.ptr, ld, q_off, k_off, v_off, b.offsets,
                                            static_cast<const int32_t *>(b.cu_dev.ptr), b.nseq, nq, nkv, hd, left, right,
                                            sinks, scale, &plan, static_cast<const float *>(table.ptr), table.ld, b.out.ptr,
                                            ldo, stream);
            return abi.attn_sink_fwd(b.qkv.ptr, ld, q_off, k_off, v_off, b.offsets,
                                     static_cast<const int32_t *>(b.cu_dev.ptr), b.nseq, nq, nkv, hd, left, right, sinks,
                                     scale, b.out.ptr, ldo, stream);
        });
    });
}

// A function's address, from a Python int.
void *address(PyObject *o) {
    void *f = PyLong_AsVoidPtr(o);
    if (!f) raise(PyExc_ValueError, "bind: not a function's address");
    return f;
}

// bind(addresses of te_quant_rows, te_rownorm_quant, te_i8_linear, te_i8_gated_linear, te_qk_rope_axes)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 5);
        void *f[5];
        for (int i = 0; i < 5; ++i) f[i] = address(a[i]);
        abi.quant_rows = reinterpret_cast<decltype(abi.quant_rows)>(f[0]);
        abi.rownorm_quant = reinterpret_cast<decltype(abi.rownorm_quant)>(f[1]);
        abi.i8_linear = reinterpret_cast<decltype(abi.i8_linear)>(f[2]);
        abi.i8_gated_linear = reinterpret_cast<decltype(abi.i8_gated_linear)>(f[3]);
        abi.qk_rope_axes = reinterpret_cast<decltype(abi.qk_rope_axes)>(f[4]);
        return TE_OK;
    });
}

// bind_attn(addresses of te_attn_sink_fwd, te_attn_relbias_fwd)
PyObject *bind_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 2);
        void *f[2];
        for (int i = 0; i < 2; ++i) f[i] = address(a[i]);
        abi.attn_sink_fwd = reinterpret_cast<decltype(abi.attn_sink_fwd)>(f[0]);
        abi.attn_relbias_fwd = reinterpret_cast<decltype(abi.attn_relbias_fwd)>(f[1]);
        return TE_OK;
    });
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"bind_attn", (PyCFunction)(void (*)(void))bind_attn, METH_FASTCALL, nullptr},
    {"quant_rows", (PyCFunction)(void (*)(void))quant_rows, METH_FASTCALL, nullptr},
    {"rownorm_quant", (PyCFunction)(void (*)(void))rownorm_quant, METH_FASTCALL, nullptr},
    {"i8_linear", (PyCFunction)(void (*)(void))i8_linear, METH_FASTCALL, nullptr},
    {"i8_gated_linear", (PyCFunction)(void (*)(void))i8_gated_linear, METH_FASTCALL, nullptr},
    {"qk_rope_axes", (PyCFunction)(void (*)(void))qk_rope_axes, METH_FASTCALL, nullptr},
    {"attn_sink_fwd", (PyCFunction)(void (*)(void))attn_span<false>, METH_FASTCALL, nullptr},
    {"attn_relbias_fwd", (PyCFunction)(void (*)(void))attn_span<true>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Argument marshalling of libtefwd's calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    K_W = PyUnicode_InternFromString("w");
    K_Y = PyUnicode_InternFromString("y");
    K_LDY = PyUnicode_InternFromString("ldy");
    K_RESIDUAL = PyUnicode_InternFromString("residual");
    K_LDR = PyUnicode_InternFromString("ldr");
    K_EPILOGUE = PyUnicode_InternFromString("epilogue");
    return PyModule_Create(&module);
}
