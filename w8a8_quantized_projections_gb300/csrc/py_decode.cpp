// Arguments of the token-by-token calls: tensors in, C ABI out.
//
// A call for a single token runs for a few microseconds on the device, less
// than its checks and its marshalling take in Python (some 60 attribute reads,
// and 4 us for 31 converted arguments): back to back, a kv_attention call took
// 22 us that way and takes 8 us here, a w4_linear call 10 and 7, kv_append with
// kv_gather 30 and 10.  So that part is compiled: each
// function checks place, type, shape and layout of its tensors (the C ABI
// receives bare pointers and cannot see lengths), allocates what the caller
// did not pass with torch's allocator, in the order of the call's stream, and
// makes one call of include/clef.h.  Nothing here synchronises, reads the
// device or keeps anything from one call for the next.
//
// Refusals are ValueErrors; a status other than CLEF_OK is raised as the
// package's ClefError.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "clef.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject *g_error = nullptr;   // ClefError

PyObject *raise(const char *call, int rc) {
    const char *text = clef_last_error();
    PyObject *detail = PyUnicode_DecodeUTF8(text, (Py_ssize_t)strlen(text), "replace");
    PyObject *value = detail ? PyObject_CallFunction(g_error, "siO", call, rc, detail) : nullptr;
    Py_XDECREF(detail);
    if (value) {
        PyErr_SetObject(g_error, value);
        Py_DECREF(value);
    }
    return nullptr;
}

// One call of the C ABI without the interpreter's lock.
#define CLEF_CALL(fn, ...)                       \
    do {                                         \
        int rc;                                  \
        Py_BEGIN_ALLOW_THREADS                   \
        rc = fn(__VA_ARGS__);                    \
        Py_END_ALLOW_THREADS                     \
        if (rc != CLEF_OK) return raise(#fn, rc); \
    } while (0)

#define CHECK(cond, ...) TORCH_CHECK_VALUE(cond, __VA_ARGS__)

// ------------------------------------------------------------ reading tensors

const Tensor &tensor(PyObject *o, const char *name) {
    CHECK(THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(), name, " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

const Tensor &on(PyObject *o, const char *name, ScalarType type, int device = -1) {
    const Tensor &t = tensor(o, name);
    CHECK(t.scalar_type() == type, name, " has dtype ", t.scalar_type(), ", expected ", type);
    CHECK(device < 0 || t.get_device() == device, name, " is on device ", (int)t.get_device(), ", other tensors on ", device);
    return t;
}

const Tensor &dense(const Tensor &t, const char *name) {
    CHECK(t.is_contiguous(), name, " must be contiguous");
    return t;
}

// Row pitch of a 2-D tensor whose rows are contiguous.
int64_t pitch(const Tensor &t, const char *name) {
    CHECK(t.dim() == 2 && (t.stride(1) == 1 || t.size(1) <= 1), name, " must be 2-D with contiguous rows");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

struct Ints {
    int32_t *at;
    int64_t n;
};

Ints ints(PyObject *o, const char *name, int device, int64_t n = -1) {
    const Tensor &t = on(o, name, ScalarType::Int, device);
    CHECK(t.dim() == 1 && (n < 0 || t.size(0) == n) && t.is_contiguous(), name, " must be contiguous int32 [",
          n < 0 ? std::string("n") : std::to_string(n), "]");
    return {(int32_t *)t.data_ptr(), t.size(0)};
}

// A pool of pages, or the two planes of a layer.
struct Pool {
    void *codes;
    float *scales;
    int64_t plane_bytes, plane_scales, pages;
    int planes, heads, page, dim, kind, device;
};

Pool pool(PyObject *co, PyObject *so, int planes) {
    Tensor c = tensor(co, "codes");
    const ScalarType type = c.scalar_type();
    CHECK(type == ScalarType::Char || type == ScalarType::Byte || type == ScalarType::Float8_e4m3fn, "codes has dtype ", type,
          ", expected int8, uint8 or float8_e4m3fn");
    const int device = c.get_device();
    Tensor s = on(so, "scales", ScalarType::Float, device);
    if (c.dim() > 5 && s.dim() == c.dim() - 2) {
        const void *at[2] = {c.data_ptr(), s.data_ptr()};
        c = c.flatten(0, -5);
        s = s.flatten(0, -3);
        CHECK(c.data_ptr() == at[0] && s.data_ptr() == at[1], "the planes of codes and scales must be evenly spaced");
    }
    CHECK(c.dim() == 5 && s.dim() == 3 && s.sizes() == c.sizes().slice(0, 3),
          "codes must be [planes][pages][heads][page][dim] and scales [planes][pages][heads]");
    const int64_t n = c.size(0), pages = c.size(1), heads = c.size(2), page = c.size(3), dim = c.size(4), tile = page * dim;
    CHECK(planes < 0 || n == planes, "codes has ", n, " planes, expected ", planes, " (a layer's keys, then its values)");
    CHECK(heads <= INT_MAX && page <= INT_MAX && dim <= INT_MAX && n <= INT_MAX, "codes' shape is out of range");
    CHECK(pages == 0 || heads == 0 || tile == 0 ||
              (c.stride(1) == heads * tile && c.stride(2) == tile && c.stride(3) == dim && c.stride(4) == 1 &&
               s.stride(1) == heads && s.stride(2) == 1),
          "each plane of codes and scales must be contiguous");
    return {c.data_ptr(),    (float *)s.data_ptr(), n > 1 ? c.stride(0) : pages * heads * tile, n > 1 ? s.stride(0) : pages * heads,
            pages,           (int)n,                (int)heads,
            (int)page,       (int)dim,              type == ScalarType::Char ? 0 : 1,
            device};
}

struct Table {
    int32_t *at;
    int64_t ld, seqs, width;
};

Table table(PyObject *o, const char *name, int device = -1) {
    const Tensor &t = on(o, name, ScalarType::Int, device);
    return {(int32_t *)t.data_ptr(), pitch(t, name), t.size(0), t.size(1)};
}

// A bf16 [tokens][heads][dim] tensor with its token and head pitch.
struct Rows {
    void *at;
    int64_t ld, ld_head, rows, heads;
};

Rows rows_of(const Tensor &t, const char *name, int64_t heads, int64_t dim) {
    CHECK(t.dim() == 3 && t.size(2) == dim && (heads < 0 || t.size(1) == heads), name, " must be [tokens][",
          heads < 0 ? std::string("heads") : std::to_string(heads), "][", dim, "], not ", t.sizes());
    CHECK(t.stride(2) == 1 || t.numel() == 0, name, " must have contiguous heads");
    const int64_t rows = t.size(0), count = t.size(1);
    return {t.data_ptr(), rows > 1 ? t.stride(0) : count * dim, count == 1 ? dim : t.stride(1), rows, count};
}

Rows rows_of(PyObject *o, const char *name, int device, int64_t heads, int64_t dim) {
    return rows_of(on(o, name, ScalarType::BFloat16, device), name, heads, dim);
}

int32_t *row_start(PyObject *o, int64_t rows, int64_t seqs, int device) {
    if (o == Py_None) {
        CHECK(rows == 0 || (seqs != 0 && rows % seqs == 0), rows, " rows for ", seqs,
              " sequences: pass row_start, or the same number for each");
        return nullptr;
    }
    return ints(o, "row_start", device, seqs + 1).at;
}

// ------------------------------------------------------------ streams, outputs

struct Stream {
    bool given;
    int device;
    cudaStream_t at;
};

Stream stream_of(PyObject *o, int device) {
    if (o == Py_None) return {false, device, c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream()};
    PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw python_error();
    void *at = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!at && PyErr_Occurred()) throw python_error();
    return {true, device, (cudaStream_t)at};
}

c10::cuda::CUDAStream external(const Stream &s) {
    const auto device = (c10::DeviceIndex)s.device;
    return s.at ? c10::cuda::getStreamFromExternal(s.at, device) : c10::cuda::getDefaultCUDAStream(device);
}

// Torch's allocator hands memory out again in the order of the stream that was
// current at its allocation, so a given stream is made the current one for it.
Tensor fresh(at::IntArrayRef shape, ScalarType type, const Stream &s) {
    const auto options = at::TensorOptions().dtype(type).device(c10::kCUDA, (c10::DeviceIndex)s.device);
    if (!s.given) return at::empty(shape, options);
    c10::cuda::CUDAStreamGuard guard(external(s));
    return at::empty(shape, options);
}

// A result that the caller passed, or a new one.
struct Result {
    Tensor own;
    PyObject *passed;

    Result(PyObject *o) : passed(o == Py_None ? nullptr : o) {}
    PyObject *object() const {
        if (!passed) return THPVariable_Wrap(own);
        Py_INCREF(passed);
        return passed;
    }
};

PyObject *pair(const Result &a, const Result &b) {
    PyObject *x = a.object(), *y = b.object();
    PyObject *t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

using Args = PyObject *const *;
#define ARGS(count)                                                                    \
    HANDLE_TH_ERRORS                                                                   \
    TORCH_CHECK_TYPE(n == (count), "expected ", (int)(count), " arguments, got ", (int)n)

// ------------------------------------------------------------ 4-bit linears

int64_t packed_columns(int64_t K) { return (K + 127) / 128 * 128; }

PyObject *quant_w4(PyObject *, Args a, Py_ssize_t n) {   // w, group, qw, sw, stream
    ARGS(5);
    const Tensor &w = on(a[0], "w", ScalarType::BFloat16);
    const int dev = w.get_device();
    const int64_t ldw = pitch(w, "w"), N = w.size(0), K = w.size(1), Kp = packed_columns(K), group = integer(a[1]);
    CHECK(group == 32 || group == 64 || group == 128, "group must be 32, 64 or 128");
    const Stream s = stream_of(a[4], dev);
    Result qw(a[2]), sw(a[3]);
    if (!qw.passed) qw.own = fresh({N, Kp / 2}, ScalarType::Byte, s);
    if (!sw.passed) sw.own = fresh({N, Kp / group}, ScalarType::BFloat16, s);
    const Tensor &q = qw.passed ? dense(on(a[2], "qw", ScalarType::Byte, dev), "qw") : qw.own;
    const Tensor &c = sw.passed ? dense(on(a[3], "sw", ScalarType::BFloat16, dev), "sw") : sw.own;
    CHECK(q.dim() == 2 && q.size(0) == N && q.size(1) == Kp / 2 && c.dim() == 2 && c.size(0) == N && c.size(1) == Kp / group,
          "qw must be [", N, "][", Kp / 2, "] and sw [", N, "][", Kp / group, "]");
    CLEF_CALL(clef_quant_w4, w.data_ptr(), N, K, ldw, (int)group, q.data_ptr(), c.data_ptr(), s.at);
    return pair(qw, sw);
    END_HANDLE_TH_ERRORS
}

PyObject *w4_linear(PyObject *, Args a, Py_ssize_t n) {   // x, qw, sw, bias, y, stream
    ARGS(6);
    const Tensor &x = on(a[0], "x", ScalarType::BFloat16);
    const int dev = x.get_device();
    const Tensor &qw = dense(on(a[1], "qw", ScalarType::Byte, dev), "qw"), &sw = dense(on(a[2], "sw", ScalarType::BFloat16, dev), "sw");
    const int64_t ldx = pitch(x, "x");
    CHECK(qw.dim() == 2 && sw.dim() == 2, "qw and sw must be 2-D");
    const int64_t M = x.size(0), K = x.size(1), N = qw.size(0), Kp = packed_columns(K), count = sw.size(1);
    CHECK(qw.size(1) * 2 == Kp, "qw has ", qw.size(1), " bytes a row, x's ", K, " columns need ", Kp / 2);
    const int64_t group = count ? Kp / count : 0;
    CHECK(sw.size(0) == N && (group == 32 || group == 64 || group == 128) && group * count == Kp, "sw has shape ", sw.sizes(),
          ": one scale for each 32, 64 or 128 of ", Kp, " weights, ", N, " rows");
    void *bias = nullptr;
    if (a[3] != Py_None) {
        const Tensor &b = dense(on(a[3], "bias", ScalarType::BFloat16, dev), "bias");
        CHECK(b.numel() == N, "bias has ", b.numel(), " values for ", N, " weight rows");
        bias = b.data_ptr();
    }
    const Stream s = stream_of(a[5], dev);
    Result out(a[4]);
    int64_t ldy = N;
    if (out.passed) {
        const Tensor &y = on(a[4], "y", ScalarType::BFloat16, dev);
        CHECK(y.dim() == 2 && y.size(0) == M && y.size(1) == N, "output has shape ", y.sizes(), ", expected [", M, ", ", N, "]");
        ldy = pitch(y, "y");
    } else {
        out.own = fresh({M, N}, ScalarType::BFloat16, s);
    }
    void *y = (out.passed ? THPVariable_Unpack(a[4]) : out.own).data_ptr();
    CLEF_CALL(clef_w4_linear, x.data_ptr(), ldx, qw.data_ptr(), sw.data_ptr(), (int)group, bias, M, N, K, y, ldy, s.at);
    return out.object();
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ cache

#define LAYER(p) (p).kind, (p).codes, (p).plane_bytes, (p).scales, (p).plane_scales, (p).pages, (p).heads, (p).page, (p).dim
#define POOL(p) (p).codes, (p).plane_bytes, (p).scales, (p).plane_scales, (p).planes, (p).pages, (p).heads, (p).page, (p).dim
#define TABLE(t) (t).at, (t).ld, (t).seqs, (t).width

PyObject *kv_append(PyObject *, Args a, Py_ssize_t n) {   // k, v, codes, scales, table, lens, row_start, stream
    ARGS(8);
    const Pool p = pool(a[2], a[3], 2);
    const Rows k = rows_of(a[0], "k", p.device, p.heads, p.dim), v = rows_of(a[1], "v", p.device, p.heads, p.dim);
    CHECK(k.rows == v.rows, "k and v differ in tokens");
    const Table t = table(a[4], "table", p.device);
    const Ints lens = ints(a[5], "lens", p.device, t.seqs);
    const int32_t *start = row_start(a[6], k.rows, t.seqs, p.device);
    const Stream s = stream_of(a[7], p.device);
    CLEF_CALL(clef_kv_append, k.at, k.ld, k.ld_head, v.at, v.ld, v.ld_head, k.rows, start, LAYER(p), TABLE(t), lens.at, s.at);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyObject *kv_gather(PyObject *, Args a, Py_ssize_t n) {   // codes, scales, table, seq, pos, k, v, stream
    ARGS(8);
    const Pool p = pool(a[0], a[1], 2);
    const Ints seq = ints(a[3], "seq", p.device), pos = ints(a[4], "pos", p.device, seq.n);
    const Table t = table(a[2], "table", p.device);
    const Stream s = stream_of(a[7], p.device);
    Result out[2] = {a[5], a[6]};
    Rows r[2];
    for (int i = 0; i < 2; ++i) {
        const char *name = i ? "v" : "k";
        if (!out[i].passed) out[i].own = fresh({seq.n, p.heads, p.dim}, ScalarType::BFloat16, s);
        r[i] = out[i].passed ? rows_of(a[5 + i], name, p.device, p.heads, p.dim) : rows_of(out[i].own, name, p.heads, p.dim);
        CHECK(r[i].rows == seq.n && r[i].ld_head == p.dim, name, " must have ", seq.n, " rows of contiguous heads");
    }
    CLEF_CALL(clef_kv_gather, LAYER(p), TABLE(t), seq.at, pos.at, seq.n, r[0].at, r[0].ld, r[1].at, r[1].ld, s.at);
    return pair(out[0], out[1]);
    END_HANDLE_TH_ERRORS
}

// q, codes, scales, table, lens, row_start, scale, causal, out, lse, stream
PyObject *kv_attention(PyObject *, Args a, Py_ssize_t n) {
    ARGS(11);
    const Pool p = pool(a[1], a[2], 2);
    const Rows q = rows_of(a[0], "q", p.device, -1, p.dim);
    CHECK(p.heads > 0 && q.heads > 0 && q.heads <= INT_MAX && q.heads % p.heads == 0, q.heads, " query heads over ", p.heads,
          " key/value heads");
    const Table t = table(a[3], "table", p.device);
    const Ints lens = ints(a[4], "lens", p.device, t.seqs);
    const int32_t *start = row_start(a[5], q.rows, t.seqs, p.device);
    double scale = std::pow((double)p.dim, -0.5);
    if (a[6] != Py_None) {
        scale = PyFloat_AsDouble(a[6]);
        if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    }
    const int causal = PyObject_IsTrue(a[7]);
    if (causal < 0) throw python_error();
    const Stream s = stream_of(a[10], p.device);
    Result out(a[8]);
    Rows o;
    if (out.passed) {
        o = rows_of(a[8], "out", p.device, q.heads, p.dim);
        CHECK(o.rows == q.rows, "out has ", o.rows, " rows, expected ", q.rows);
        // tokens of heads, or heads of tokens: either way the inner run has to fit between two of the outer
        CHECK(q.rows == 0 || o.ld >= (q.heads - 1) * o.ld_head + p.dim ||
                  (o.ld_head >= (q.rows - 1) * o.ld + p.dim && o.ld >= p.dim),
              "out's rows overlap");
    } else {
        out.own = fresh({q.rows, q.heads, p.dim}, ScalarType::BFloat16, s);
        o = {out.own.data_ptr(), q.heads * p.dim, p.dim, q.rows, q.heads};
    }
    float *lse = nullptr;
    if (a[9] != Py_None) {
        const Tensor &l = dense(on(a[9], "lse", ScalarType::Float, p.device), "lse");
        CHECK(l.dim() == 2 && l.size(0) == q.rows && l.size(1) == q.heads, "lse must be [", q.rows, "][", q.heads, "]");
        lse = (float *)l.data_ptr();
    }
    int64_t need = 0;
    const int64_t top = std::min<int64_t>(t.width * p.page, INT_MAX);
    CLEF_CALL(clef_kv_attention_workspace, q.rows, start != nullptr, t.seqs, (int)q.heads, p.heads, p.dim, top, &need);
    Tensor ws;
    if (need) ws = fresh({need}, ScalarType::Byte, s);
    CLEF_CALL(clef_kv_attention, q.at, q.ld, q.ld_head, q.rows, start, (int)q.heads, LAYER(p), TABLE(t), lens.at, (float)scale,
              causal, o.at, o.ld, o.ld_head, lse, need ? ws.data_ptr() : nullptr, need, s.at);
    return out.object();
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ pages

PyObject *kv_reserve(PyObject *, Args a, Py_ssize_t n) {   // table, lens, refs, grow, page, stream, row_start
    ARGS(7);
    const Table t = table(a[0], "table");
    const int dev = THPVariable_Unpack(a[0]).get_device();
    const Ints lens = ints(a[1], "lens", dev, t.seqs), refs = ints(a[2], "refs", dev), grow = ints(a[3], "grow", dev, t.seqs);
    const Stream s = stream_of(a[5], dev);
    int32_t *rows = a[6] == Py_None ? nullptr : ints(a[6], "row_start", dev, t.seqs + 1).at;
    CLEF_CALL(clef_kv_reserve_rows, TABLE(t), lens.at, refs.at, refs.n, (int)integer(a[4]), grow.at, rows, s.at);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyObject *kv_fork(PyObject *, Args a, Py_ssize_t n) {   // codes, scales, table, lens, refs, src, dst, stream
    ARGS(8);
    const Pool p = pool(a[0], a[1], -1);
    const Table t = table(a[2], "table", p.device);
    const Ints lens = ints(a[3], "lens", p.device, t.seqs), refs = ints(a[4], "refs", p.device, p.pages),
               src = ints(a[5], "src", p.device), dst = ints(a[6], "dst", p.device, src.n);
    const Stream s = stream_of(a[7], p.device);
    const Tensor scratch = fresh({2 * src.n}, ScalarType::Int, s);
    CLEF_CALL(clef_kv_fork, POOL(p), TABLE(t), lens.at, refs.at, src.at, dst.at, src.n, (int32_t *)scratch.data_ptr(), s.at);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyObject *kv_free(PyObject *, Args a, Py_ssize_t n) {   // table, lens, refs, seqs, page, stream
    ARGS(6);
    const Table t = table(a[0], "table");
    const int dev = THPVariable_Unpack(a[0]).get_device();
    const Ints lens = ints(a[1], "lens", dev, t.seqs), refs = ints(a[2], "refs", dev), list = ints(a[3], "seqs", dev);
    const Stream s = stream_of(a[5], dev);
    CLEF_CALL(clef_kv_free, TABLE(t), lens.at, refs.at, refs.n, (int)integer(a[4]), list.at, list.n, s.at);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyObject *kv_compact(PyObject *, Args a, Py_ssize_t n) {   // codes, scales, table, lens, refs, table_out, refs_out, stream
    ARGS(8);
    const Pool p = pool(a[0], a[1], -1);
    PyObject *to = a[5] == Py_None ? a[2] : a[5], *ro = a[6] == Py_None ? a[4] : a[6];
    const Table t = table(a[2], "table", p.device), t_out = table(to, "table_out", p.device);
    const Ints lens = ints(a[3], "lens", p.device, t.seqs), refs = ints(a[4], "refs", p.device, p.pages),
               refs_out = ints(ro, "refs_out", p.device, p.pages);
    CHECK(t_out.seqs == t.seqs && t_out.width == t.width, "table_out has another shape than table");
    const Stream s = stream_of(a[7], p.device);
    Result live(Py_None);
    live.own = fresh({1}, ScalarType::Int, s);
    if (p.pages == 0) {   // an empty call writes nothing
        c10::cuda::CUDAStreamGuard guard(external(s));
        live.own.zero_();
    }
    const Tensor scratch = fresh({3 * p.pages + 1}, ScalarType::Int, s);
    CLEF_CALL(clef_kv_compact, POOL(p), TABLE(t), lens.at, refs.at, t_out.at, t_out.ld, refs_out.at,
              (int32_t *)live.own.data_ptr(), (int32_t *)scratch.data_ptr(), s.at);
    return live.object();
    END_HANDLE_TH_ERRORS
}

PyObject *kv_copy_pages(PyObject *, Args a, Py_ssize_t n) {   // codes, scales, src, dst, stream
    ARGS(5);
    const Pool p = pool(a[0], a[1], -1);
    const Ints src = ints(a[2], "src", p.device), dst = ints(a[3], "dst", p.device, src.n);
    const Stream s = stream_of(a[4], p.device);
    CLEF_CALL(clef_kv_copy_pages, POOL(p), src.at, dst.at, src.n, s.at);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}

PyMethodDef methods[] = {METHOD(quant_w4),   METHOD(w4_linear),  METHOD(kv_append),     METHOD(kv_gather),
                         METHOD(kv_attention), METHOD(kv_reserve), METHOD(kv_fork),     METHOD(kv_free),
                         METHOD(kv_compact), METHOD(kv_copy_pages), {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "clef_decode", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_clef_decode(void) { return PyModule_Create(&module); }
