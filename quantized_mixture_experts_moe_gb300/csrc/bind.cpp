// Argument marshalling of the calls around the experts (norms, routing, FP8
// products, the experts' products for training, 4-bit products) between torch tensors and the C ABI: checks, output allocation and
// one call each, no arithmetic.  The kernels take a few microseconds for a
// single token; marshalled from Python through ctypes a call took 13 to 19 us
// of host time.  binding.py wraps these functions and documents them.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/qmoe.h"

namespace {

PyObject* qmoe_error = nullptr;  // binding.QmoeError

// An exception that is already set in Python.
struct PythonError {};

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw PythonError{};
}
[[noreturn]] void bad(const std::string& what) { refuse(PyExc_ValueError, what); }

void check(int rc, const char* name) {
    if (rc == 0) return;
    std::ostringstream s;
    s << name << " failed: " << rc << " (" << qmoe_status_str(rc) << ")";
    refuse(qmoe_error, s.str());
}

std::string shape_str(const at::Tensor& t) {
    std::ostringstream s;
    s << t.sizes() << " of " << t.scalar_type();
    return s.str();
}

// ------------------------------------------------------------------ arguments

struct Args {
    PyObject* const* v;
    Py_ssize_t n;
    const char* name;
    Args(PyObject* const* v_, Py_ssize_t n_, Py_ssize_t want, const char* name_) : v(v_), n(n_), name(name_) {
        if (n != want) refuse(PyExc_TypeError, std::string(name) + ": wrong number of arguments");
    }
    bool none(int i) const { return v[i] == Py_None; }
    // The device of the arguments that lie on one: launches go to it.
    std::optional<at::Device> device() const {
        std::optional<at::Device> one;
        for (Py_ssize_t i = 0; i < n; ++i) {
            // what is told by its type alone first: the tensors' check is a slow one for all else (0.3 us a call)
            if (v[i] == Py_None || PyFloat_CheckExact(v[i]) || PyLong_Check(v[i]) || !THPVariable_Check(v[i])) continue;
            const at::Device d = THPVariable_Unpack(v[i]).device();
            if (!d.is_cuda()) continue;
            if (one && *one != d) {
                std::ostringstream s;
                s << "qmoe kernels take tensors of one device, got " << *one << " and " << d;
                refuse(qmoe_error, s.str());
            }
            one = d;
        }
        return one;
    }
    const at::Tensor& tensor(int i) const {
        if (!THPVariable_Check(v[i])) refuse(PyExc_TypeError, std::string(name) + ": expected a torch.Tensor");
        return THPVariable_Unpack(v[i]);
    }
    const at::Tensor* maybe(int i) const { return none(i) ? nullptr : &tensor(i); }
    double number(int i) const {
        const double d = PyFloat_AsDouble(v[i]);
        if (d == -1.0 && PyErr_Occurred()) throw PythonError{};
        return d;
    }
    int64_t whole(int i) const {
        const long long x = PyLong_AsLongLong(v[i]);
        if (x == -1 && PyErr_Occurred()) throw PythonError{};
        return x;
    }
    bool truth(int i) const {
        const int x = PyObject_IsTrue(v[i]);
        if (x < 0) throw PythonError{};
        return x != 0;
    }
    at::ScalarType dtype(int i, at::ScalarType otherwise) const {
        if (none(i)) return otherwise;
        if (!THPDtype_Check(v[i])) refuse(PyExc_TypeError, std::string(name) + ": expected a torch.dtype");
        return reinterpret_cast<THPDtype*>(v[i])->scalar_type;
    }
};

int code_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return QMOE_F32;
        case at::kBFloat16:
        case at::kShort: return QMOE_BF16;  // int16: bf16 bits
        case at::kHalf: return QMOE_F16;
        default: break;
    }
    std::ostringstream s;
    s << "expected float32, bfloat16 or float16, got " << t;
    bad(s.str());
}

void on_device(const at::Tensor& t) {
    if (!t.is_cuda()) refuse(qmoe_error, "qmoe kernels take device tensors");
}

// A matrix's pointer and row stride.
struct Rows {
    void* p = nullptr;
    int64_t ld = 0;
};
Rows rows_of(const at::Tensor& t, int64_t T, int64_t H) {
    if (t.dim() != 2 || t.size(0) != T || t.size(1) != H) {
        std::ostringstream s;
        s << "expected a tensor of shape [" << T << ", " << H << "], got " << shape_str(t);
        bad(s.str());
    }
    on_device(t);
    if (t.stride(1) != 1 && H > 1) refuse(qmoe_error, "qmoe kernels take rows of contiguous columns");
    int64_t ld = t.stride(0);
    if (ld < H) {
        if (T > 1) refuse(qmoe_error, "qmoe kernels take rows that do not overlap");
        ld = H;
    }
    return {t.data_ptr(), ld};
}
void matrix(const at::Tensor& t, const char* what) {
    if (t.dim() != 2) bad(std::string(what) + ": expected a tensor of shape [rows, cols], got " + shape_str(t));
}

template <typename T>
T* vec_of(const at::Tensor* t, int64_t n, at::ScalarType type) {
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->numel() != n) {
        std::ostringstream s;
        s << "expected " << n << " values of " << type << ", got " << shape_str(*t);
        bad(s.str());
    }
    on_device(*t);
    if (!t->is_contiguous()) refuse(qmoe_error, "qmoe kernels take contiguous tensors");
    return static_cast<T*>(t->data_ptr());
}
float* floats(const at::Tensor* t, int64_t n) { return vec_of<float>(t, n, at::kFloat); }

struct Gate {
    int mode = QMOE_GATE_NONE;
    void* p = nullptr;
    int64_t ld = 0;
};
Gate gate_of(const at::Tensor* g, int64_t T, int64_t H, at::ScalarType block) {
    if (!g) return {};
    const auto s = g->sizes();
    const bool two = s.size() == 2;
    const bool fp32 = g->scalar_type() == at::kFloat;
    if ((s.size() == 1 && s[0] == T) || (two && s[0] == T && s[1] == 1 && fp32)) return {QMOE_GATE_ROW, floats(g, T), 0};
    if (two && s[0] == T && s[1] == H && g->scalar_type() == block) {
        const Rows r = rows_of(*g, T, H);
        return {QMOE_GATE_FULL, r.p, r.ld};
    }
    if ((s.size() == 1 && s[0] == H) || (two && s[0] == 1 && s[1] == H)) return {QMOE_GATE_COL, floats(g, H), 0};
    bad("a gate is fp32 [T, 1], [T], [1, H] or [H], or [T, H] of the block's type; got " + shape_str(*g));
}

// ------------------------------------------------------------------ outputs

at::Tensor make(at::IntArrayRef size, at::ScalarType type, const at::Tensor& like) {
    // past the dispatcher: half the host time of an output
    return at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
}
// Small outputs of one call, in one allocation: each on a 256-byte boundary.
struct Pieces {
    struct Piece {
        std::array<int64_t, 2> size;
        int dims;
        at::ScalarType type;
        int64_t at;
    };
    std::array<Piece, 6> piece;
    int n = 0;
    int64_t bytes = 0;

    int add(int64_t a, int64_t b, int dims, at::ScalarType type) {
        piece[n] = {{a, b}, dims, type, bytes};
        bytes += (a * b * 4 + 255) / 256 * 256;  // 32-bit types
        return n++;
    }
    std::array<at::Tensor, 6> allocate(const at::Tensor& like) const {
        const at::Tensor block = make({bytes / 4}, at::kFloat, like);
        std::array<at::Tensor, 6> out;
        for (int i = 0; i < n; ++i) {
            out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(block.storage()), block.key_set(),
                                                              at::scalarTypeToTypeMeta(piece[i].type));
            c10::TensorImpl* const t = out[i].unsafeGetTensorImpl();
            t->set_storage_offset(piece[i].at / 4);
            t->set_sizes_contiguous(at::IntArrayRef(piece[i].size.data(), piece[i].dims));
        }
        return out;
    }
};
qmoe_stream_t stream_of(const at::Tensor& t) {
    return reinterpret_cast<qmoe_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

struct Workspace {
    at::Tensor held;
    void* p = nullptr;
    size_t n = 0;
    Workspace(size_t need, const at::Tensor* given, const at::Tensor& like) {
        if (given) {
            on_device(*given);
            if (!given->is_contiguous()) refuse(qmoe_error, "qmoe kernels take contiguous tensors");
            held = *given;
        } else {
            held = make({(int64_t)(need > 256 ? need : 256)}, at::kByte, like);
        }
        p = held.data_ptr();
        n = held.nbytes();
    }
};

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw PythonError{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}
void* at_of(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* f32_of(const at::Tensor& t) { return static_cast<float*>(at_of(t)); }

// ------------------------------------------------------------------ norms

PyObject* norm_pre(const Args& a) {  // x, w, eps, out_dtype
    const at::Tensor &x = a.tensor(0), &w = a.tensor(1);
    matrix(x, "norm_pre");
    const int64_t T = x.size(0), H = x.size(1);
    const auto st = x.scalar_type(), bt = a.dtype(3, st);
    const Rows xr = rows_of(x, T, H);
    const int sc = code_of(st), bc = code_of(bt);
    const float* wp = floats(&w, H);
    const at::Tensor n = make({T, H}, bt, x), rstd = make({T}, at::kFloat, x);
    check(qmoe_norm_pre(T, H, sc, bc, xr.p, xr.ld, wp, (float)a.number(2), n.data_ptr(), H, f32_of(rstd), stream_of(x)),
          "qmoe_norm_pre");
    return tuple_of({n, rstd});
}

PyObject* norm_pre_backward(const Args& a) {  // dn, x, rstd, w, dres, ws
    const at::Tensor &dn = a.tensor(0), &x = a.tensor(1), *dres = a.maybe(4);
    matrix(x, "norm_pre_backward");
    const int64_t T = x.size(0), H = x.size(1);
    const auto st = x.scalar_type();
    if (dres && dres->scalar_type() != st) bad("dres has x's type");
    const Rows xr = rows_of(x, T, H), dnr = rows_of(dn, T, H), dr = dres ? rows_of(*dres, T, H) : Rows{};
    const int sc = code_of(st), bc = code_of(dn.scalar_type());
    const float *rp = floats(&a.tensor(2), T), *wp = floats(&a.tensor(3), H);
    const at::Tensor dx = make({T, H}, st, x), dw = make({H}, at::kFloat, x);
    const Workspace ws(qmoe_norm_bwd_workspace_bytes(T, H), a.maybe(5), x);
    check(qmoe_norm_pre_backward(T, H, sc, bc, dnr.p, dnr.ld, xr.p, xr.ld, rp, wp, dr.p, dr.ld, dx.data_ptr(), H,
                                 f32_of(dw), ws.p, ws.n, stream_of(x)),
          "qmoe_norm_pre_backward");
    return tuple_of({dx, dw});
}

PyObject* norm_post(const Args& a) {  // r, y, w, gate, alpha, w_next, eps
    const at::Tensor &r = a.tensor(0), &y = a.tensor(1), *w = a.maybe(2), *gate = a.maybe(3), *wn = a.maybe(5);
    matrix(y, "norm_post");
    const int64_t T = y.size(0), H = y.size(1);
    const auto st = r.scalar_type(), bt = y.scalar_type();
    const Rows rr = rows_of(r, T, H), yr = rows_of(y, T, H);
    const int sc = code_of(st), bc = code_of(bt);
    const Gate g = gate_of(gate, T, H, bt);
    const float *wp = floats(w, H), *wnp = floats(wn, H);
    at::Tensor out = make({T, H}, st, y), n, rstd, rstd_next;
    if (w) rstd = make({T}, at::kFloat, y);
    if (wn) {
        n = make({T, H}, bt, y);
        rstd_next = make({T}, at::kFloat, y);
    }
    check(qmoe_norm_post(T, H, sc, bc, rr.p, rr.ld, yr.p, yr.ld, wp, g.mode, g.p, g.ld, (float)a.number(4), wnp,
                         (float)a.number(6), out.data_ptr(), H, at_of(n), H, f32_of(rstd), f32_of(rstd_next),
                         stream_of(y)),
          "qmoe_norm_post");
    return tuple_of({out, n, rstd, rstd_next});
}

PyObject* norm_post_backward(const Args& a) {  // dout, y, w, rstd, gate, alpha, dn, out, w_next, rstd_next, ws
    const at::Tensor *dout = a.maybe(0), &y = a.tensor(1), *w = a.maybe(2), *rstd = a.maybe(3), *gate = a.maybe(4),
                     *dn = a.maybe(6), *out = a.maybe(7), *wn = a.maybe(8), *rn = a.maybe(9);
    matrix(y, "norm_post_backward");
    const int64_t T = y.size(0), H = y.size(1);
    const auto bt = y.scalar_type();
    if (!dout && !dn) bad("norm_post_backward needs dout or dn");
    if (w && !rstd) bad("w needs rstd");
    if (dn && (!out || !wn || !rn)) bad("dn needs out, w_next and rstd_next");
    if (dn && (dn->scalar_type() != bt || (dout && out->scalar_type() != dout->scalar_type())))
        bad("dn has y's type, and out dout's");
    const auto st = dout ? dout->scalar_type() : out->scalar_type();
    const Rows yr = rows_of(y, T, H), dor = dout ? rows_of(*dout, T, H) : Rows{}, dnr = dn ? rows_of(*dn, T, H) : Rows{},
               outr = dn ? rows_of(*out, T, H) : Rows{};
    const int sc = code_of(st), bc = code_of(bt);
    const Gate g = gate_of(gate, T, H, bt);
    const float *wp = floats(w, H), *rp = w ? floats(rstd, T) : nullptr, *wnp = dn ? floats(wn, H) : nullptr,
                *rnp = dn ? floats(rn, T) : nullptr;
    at::Tensor dr = make({T, H}, st, y), dy = make({T, H}, bt, y), dw, dgate, dwn;
    if (w) dw = make({H}, at::kFloat, y);
    if (gate) dgate = make(gate->sizes(), gate->scalar_type(), y);
    if (dn) dwn = make({H}, at::kFloat, y);
    if (T == 0) {  // no rows (and no pointers to tell what was given): the sums are zero
        for (at::Tensor* t : {&dw, &dgate, &dwn})
            if (t->defined()) t->zero_();
        return tuple_of({dr, dy, dw, dgate, dwn});
    }
    const Workspace ws(qmoe_norm_bwd_workspace_bytes(T, H), a.maybe(10), y);
    check(qmoe_norm_post_backward(T, H, sc, bc, dor.p, dor.ld, yr.p, yr.ld, wp, rp, g.mode, g.p, g.ld,
                                  (float)a.number(5), dnr.p, dnr.ld, outr.p, outr.ld, wnp, rnp, dr.data_ptr(), H,
                                  dy.data_ptr(), H, f32_of(dw), at_of(dgate), H, f32_of(dwn), ws.p, ws.n, stream_of(y)),
          "qmoe_norm_post_backward");
    return tuple_of({dr, dy, dw, dgate, dwn});
}

// ------------------------------------------------------------------ routing

PyObject* route_topk(const Args& a) {  // logits, k, bias, mask, renorm, scale, coef, ws
    const at::Tensor &lg = a.tensor(0), *mask = a.maybe(3);
    matrix(lg, "route_topk");
    const int64_t T = lg.size(0), E = lg.size(1), k = a.whole(1);
    if (k < 0 || k > 1 << 20 || E > 1 << 20) check(QMOE_ERR_UNSUPPORTED, "qmoe_route_topk");
    const Rows r = rows_of(lg, T, E);
    const int code = code_of(lg.scalar_type());
    const float* bias = floats(a.maybe(2), E);
    const uint8_t* mp = nullptr;
    if (mask)
        mp = mask->scalar_type() == at::kBool ? vec_of<uint8_t>(mask, T, at::kBool) : vec_of<uint8_t>(mask, T, at::kByte);
    const bool stats = !a.none(6);
    Pieces pieces;
    pieces.add(T, k, 2, at::kInt);
    pieces.add(T, k, 2, at::kFloat);
    pieces.add(T, 1, 1, at::kFloat);
    if (stats) {
        pieces.add(E + 1, 1, 1, at::kInt);
        pieces.add(E, 1, 1, at::kFloat);
        pieces.add(1, 1, 1, at::kFloat);
    }
    const auto [ids, w, lse, counts, probs, loss] = pieces.allocate(lg);
    if (!stats) {
        check(qmoe_route_topk(T, (int)E, (int)k, code, r.p, r.ld, bias, mp, a.truth(4), (float)a.number(5),
                              static_cast<int32_t*>(ids.data_ptr()), f32_of(w), f32_of(lse), 0.f, nullptr, nullptr,
                              nullptr, nullptr, 0, stream_of(lg)),
              "qmoe_route_topk");
    } else {
        const Workspace ws(qmoe_route_workspace_bytes(T, (int)E), a.maybe(7), lg);
        check(qmoe_route_topk(T, (int)E, (int)k, code, r.p, r.ld, bias, mp, a.truth(4), (float)a.number(5),
                              static_cast<int32_t*>(ids.data_ptr()), f32_of(w), f32_of(lse), (float)a.number(6),
                              static_cast<int32_t*>(counts.data_ptr()), f32_of(probs), f32_of(loss), ws.p, ws.n,
                              stream_of(lg)),
              "qmoe_route_topk");
    }
    return tuple_of({ids, w, lse, counts, probs, loss});
}

PyObject* route_topk_backward(const Args& a) {  // logits, ids, w, lse, counts, renorm, scale, coef, dw, dloss
    const at::Tensor &lg = a.tensor(0), &ids = a.tensor(1), *dw = a.maybe(8), *dloss = a.maybe(9);
    matrix(lg, "route_topk_backward");
    matrix(ids, "route_topk_backward");
    const int64_t T = lg.size(0), E = lg.size(1), k = ids.size(1);
    if (!dw && !dloss) bad("route_topk_backward needs dw or dloss");
    if (dloss && a.none(4)) bad("dloss needs a routing made with coef");
    const Rows r = rows_of(lg, T, E);
    const int code = code_of(lg.scalar_type());
    const at::Tensor dl = make({T, E}, lg.scalar_type(), lg);
    if (T == 0) return wrap(dl);
    check(qmoe_route_topk_backward(T, (int)E, (int)k, code, r.p, r.ld, vec_of<int32_t>(&ids, T * k, at::kInt),
                                   floats(&a.tensor(2), T * k), floats(&a.tensor(3), T), a.truth(5), (float)a.number(6),
                                   floats(dw, T * k), a.none(7) ? 0.f : (float)a.number(7),
                                   vec_of<int32_t>(a.maybe(4), E + 1, at::kInt), floats(dloss, 1), dl.data_ptr(), E,
                                   stream_of(lg)),
          "qmoe_route_topk_backward");
    return wrap(dl);
}

// ------------------------------------------------------------------ FP8

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

// A new tensor's own sizes and strides within what was allocated (a view of it costs a microsecond).
void lay_out(const at::Tensor& t, at::IntArrayRef sizes, at::IntArrayRef strides) {
    t.unsafeGetTensorImpl()->set_sizes_and_strides(sizes, strides);
}
// Uninitialised codes [rows, cols] whose rows start on 16-byte boundaries.
at::Tensor codes(int64_t rows, int64_t cols, const at::Tensor& like) {
    const at::Tensor q = make({rows, up16(cols)}, at::kFloat8_e4m3fn, like);
    if (up16(cols) != cols) lay_out(q, {rows, cols}, {up16(cols), 1});
    return q;
}
// Uninitialised scales [rows, blocks] that lie block by block.
at::Tensor scales(int64_t rows, int64_t blocks, const at::Tensor& like) {
    const at::Tensor s = make({blocks, rows}, at::kFloat, like);
    lay_out(s, {rows, blocks}, {1, rows});
    return s;
}
uint8_t* bytes_of(const at::Tensor& t) { return static_cast<uint8_t*>(at_of(t)); }

PyObject* fp8_quant_rows(const Args& a) {  // x
    const at::Tensor& x = a.tensor(0);
    matrix(x, "fp8_quant_rows");
    const int64_t T = x.size(0), K = x.size(1);
    const Rows r = rows_of(x, T, K);
    const int code = code_of(x.scalar_type());
    const at::Tensor q = codes(T, K, x), s = scales(T, blocks_of(K), x);
    check(qmoe_fp8_quant_rows(T, K, code, r.p, r.ld, bytes_of(q), up16(K), f32_of(s), stream_of(x)),
          "qmoe_fp8_quant_rows");
    return tuple_of({q, s});
}

PyObject* fp8_quant_cols(const Args& a) {  // x, rows_too
    const at::Tensor& x = a.tensor(0);
    matrix(x, "fp8_quant_cols");
    const int64_t T = x.size(0), K = x.size(1);
    const Rows r = rows_of(x, T, K);
    const int code = code_of(x.scalar_type());
    const at::Tensor qt = codes(K, T, x), st = scales(K, blocks_of(T), x);
    at::Tensor q, s;
    if (a.truth(1)) {
        q = codes(T, K, x);
        s = scales(T, blocks_of(K), x);
    }
    check(qmoe_fp8_quant_cols(T, K, code, r.p, r.ld, bytes_of(qt), up16(T), f32_of(st), bytes_of(q), up16(K), f32_of(s),
                              stream_of(x)),
          "qmoe_fp8_quant_cols");
    return q.defined() ? tuple_of({qt, st, q, s}) : tuple_of({qt, st});
}

PyObject* fp8_quant_blocks(const Args& a) {  // w, transposed
    const at::Tensor& w = a.tensor(0);
    matrix(w, "fp8_quant_blocks");
    const int64_t N = w.size(0), K = w.size(1);
    const Rows r = rows_of(w, N, K);
    const int code = code_of(w.scalar_type());
    const at::Tensor q = codes(N, K, w), s = make({blocks_of(N), blocks_of(K)}, at::kFloat, w);
    at::Tensor qt;
    if (a.truth(1)) qt = codes(K, N, w);
    check(qmoe_fp8_quant_blocks(N, K, code, r.p, r.ld, bytes_of(q), up16(K), bytes_of(qt), up16(N), f32_of(s),
                                stream_of(w)),
          "qmoe_fp8_quant_blocks");
    return qt.defined() ? tuple_of({q, s, qt}) : tuple_of({q, s});
}

qmoe_fp8_mat mat_of(const at::Tensor& q, const at::Tensor& s) {
    matrix(q, "codes");
    matrix(s, "scales");
    const int64_t rows = q.size(0), K = q.size(1);
    if (q.scalar_type() != at::kFloat8_e4m3fn && q.scalar_type() != at::kByte)
        bad("expected float8_e4m3fn or uint8 codes, got " + shape_str(q));
    const bool own = s.size(0) == rows;
    if (s.scalar_type() != at::kFloat || s.size(1) != blocks_of(K) || (!own && s.size(0) != blocks_of(rows))) {
        std::ostringstream m;
        m << "expected fp32 scales [" << rows << " or " << blocks_of(rows) << ", " << blocks_of(K) << "], got "
          << shape_str(s);
        bad(m.str());
    }
    on_device(s);
    const Rows r = rows_of(q, rows, K);
    // the stride of a single row is not used
    return {static_cast<const uint8_t*>(r.p), rows == 1 ? up16(r.ld) : r.ld, f32_of(s), s.stride(0), s.stride(1),
            own ? 1 : 128, 0};
}
int32_t* status_of(const at::Tensor& t) { return vec_of<int32_t>(&t, 1, at::kInt); }

PyObject* fp8_matmul(const Args& a) {  // a_q, a_s, b_q, b_s, out_dtype, dev_status
    const at::Tensor &aq = a.tensor(0), &bq = a.tensor(2);
    const qmoe_fp8_mat ma = mat_of(aq, a.tensor(1)), mb = mat_of(bq, a.tensor(3));
    const int64_t M = aq.size(0), K = aq.size(1), N = bq.size(0);
    if (bq.size(1) != K) bad("the reduction lengths differ: " + shape_str(aq) + " and " + shape_str(bq));
    const auto ct = a.dtype(4, at::kBFloat16);
    const int code = code_of(ct);
    const at::Tensor c = make({M, N}, ct, aq);
    check(qmoe_fp8_matmul(M, N, K, &ma, &mb, c.data_ptr(), code, N, status_of(a.tensor(5)), stream_of(aq)),
          "qmoe_fp8_matmul");
    return wrap(c);
}

PyObject* fp8_linear(const Args& a) {  // x, w_q, w_s, out_dtype, dev_status, ws
    const at::Tensor &x = a.tensor(0), &wq = a.tensor(1);
    matrix(x, "fp8_linear");
    const qmoe_fp8_mat w = mat_of(wq, a.tensor(2));
    const int64_t T = x.size(0), K = x.size(1), N = wq.size(0);
    if (wq.size(1) != K) bad("the reduction lengths differ: " + shape_str(x) + " and " + shape_str(wq));
    const Rows r = rows_of(x, T, K);
    const auto yt = a.dtype(3, x.scalar_type());
    const int xc = code_of(x.scalar_type()), yc = code_of(yt);
    const at::Tensor y = make({T, N}, yt, x);
    const Workspace ws(qmoe_fp8_linear_workspace_bytes(T, K), a.maybe(5), x);
    check(qmoe_fp8_linear(T, N, K, xc, r.p, r.ld, &w, y.data_ptr(), yc, N, status_of(a.tensor(4)), ws.p, ws.n,
                          stream_of(x)),
          "qmoe_fp8_linear");
    return wrap(y);
}

PyObject* fp8_linear_backward(const Args& a) {  // dy, x, wt_q, w_s, dev_status
    const at::Tensor &dy = a.tensor(0), &x = a.tensor(1), &wt = a.tensor(2);
    matrix(dy, "fp8_linear_backward");
    matrix(x, "fp8_linear_backward");
    matrix(wt, "fp8_linear_backward");
    const int64_t T = dy.size(0), N = dy.size(1), K = x.size(1);
    if (x.size(0) != T || wt.size(0) != K || wt.size(1) != N)
        bad("dy [T, N], x [T, K] and wt_q [K, N] do not go together: " + shape_str(dy) + ", " + shape_str(x) + " and " +
            shape_str(wt));
    on_device(dy);
    const at::Tensor dx = make({T, K}, dy.scalar_type(), dy);
    if (T == 0) return tuple_of({dx, at::zeros({N, K}, at::TensorOptions().dtype(at::kFloat).device(dy.device()))});
    const qmoe_fp8_mat w = mat_of(wt, a.tensor(3).t());
    const Rows yr = rows_of(dy, T, N), xr = rows_of(x, T, K);
    const int yc = code_of(dy.scalar_type()), xc = code_of(x.scalar_type());
    int32_t* const status = status_of(a.tensor(4));
    const qmoe_stream_t st = stream_of(dy);
    const at::Tensor dw = make({N, K}, at::kFloat, dy);
    // codes and scales of dy^T, dy and x^T, in one allocation
    const int64_t rows[3] = {N, T, K}, cols[3] = {T, N, T};
    int64_t at[6], bytes = 0;
    for (int i = 0; i < 3; ++i) {
        at[2 * i] = bytes;
        bytes += (rows[i] * up16(cols[i]) + 255) / 256 * 256;
        at[2 * i + 1] = bytes;
        bytes += (rows[i] * blocks_of(cols[i]) * 4 + 255) / 256 * 256;
    }
    const at::Tensor held = make({bytes}, at::kByte, dy);
    uint8_t* const base = static_cast<uint8_t*>(held.data_ptr());
    qmoe_fp8_mat m[3];
    float* s[3];
    for (int i = 0; i < 3; ++i) {
        s[i] = reinterpret_cast<float*>(base + at[2 * i + 1]);
        m[i] = {base + at[2 * i], up16(cols[i]), s[i], 1, rows[i], 1, 0};
    }
    check(qmoe_fp8_quant_cols(T, N, yc, yr.p, yr.ld, base + at[0], m[0].ld, s[0], base + at[2], m[1].ld, s[1], st),
          "qmoe_fp8_quant_cols");
    check(qmoe_fp8_quant_cols(T, K, xc, xr.p, xr.ld, base + at[4], m[2].ld, s[2], nullptr, 0, nullptr, st),
          "qmoe_fp8_quant_cols");
    check(qmoe_fp8_matmul(T, K, N, &m[1], &w, dx.data_ptr(), yc, K, status, st), "qmoe_fp8_matmul");
    check(qmoe_fp8_matmul(N, K, T, &m[0], &m[2], dw.data_ptr(), QMOE_F32, K, status, st), "qmoe_fp8_matmul");
    return tuple_of({dx, dw});
}

// ------------------------------------------------------------------ the experts' products

// Weights [E, N, K] (or [N, K], one expert) of contiguous columns.
struct Experts {
    void* p = nullptr;
    int64_t E = 1, N = 0, K = 0, ld = 0, stride = 0;
};
Experts experts_of(const at::Tensor& w, const char* what) {
    if (w.dim() != 3) bad(std::string(what) + ": expected weights of shape [experts, outputs, inputs], got " + shape_str(w));
    on_device(w);
    Experts m = {w.data_ptr(), w.size(0), w.size(1), w.size(2), w.stride(1), w.stride(0)};
    if (m.E > 1 << 20) check(QMOE_ERR_UNSUPPORTED, what);
    if (w.stride(2) != 1 && m.K > 1) refuse(qmoe_error, "qmoe kernels take rows of contiguous columns");
    if (m.ld < m.K) {
        if (m.N > 1) refuse(qmoe_error, "qmoe kernels take rows that do not overlap");
        m.ld = m.K;
    }
    if (m.stride < m.ld * (m.N - 1) + m.K) {
        if (m.E > 1) refuse(qmoe_error, "qmoe kernels take rows that do not overlap");
        m.stride = m.ld * m.N;
    }
    return m;
}
bool in_pieces(const void* p, int64_t rows, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows == 1 || ld % 8 == 0);
}
size_t copy_of(const Rows& r, int64_t rows, int64_t cols) {
    return in_pieces(r.p, rows, r.ld) ? 0 : qmoe_expert_copy_bytes(rows, cols);
}
size_t copy_of(const Experts& m) {
    return in_pieces(m.p, m.N, m.ld) && (m.E == 1 || m.stride % 8 == 0) ? 0 : qmoe_expert_copy_bytes(m.E * m.N, m.K);
}
// What a call needs of the workspace is mostly nothing: then none is made.
struct MaybeWorkspace {
    std::optional<Workspace> held;
    void* p = nullptr;
    size_t n = 0;
    MaybeWorkspace(size_t need, const at::Tensor* given, const at::Tensor& like) {
        if (!given && !need) return;
        held.emplace(need, given, like);
        p = held->p;
        n = held->n;
    }
};
int same_type(const at::Tensor& a, const at::Tensor& b, const char* what) {
    if (a.scalar_type() != b.scalar_type()) bad(std::string(what) + " have one type, got " + shape_str(a) + " and " + shape_str(b));
    const int code = code_of(a.scalar_type());
    if (code == QMOE_F32) bad(std::string(what) + " are of bfloat16 or float16");
    return code;
}
// The rows in expert order and where they lie in x.
struct Gathered {
    int64_t P, rows;
    Rows x;
    const int32_t* pairs = nullptr;
    int k = 1;
};
Gathered gathered(const at::Tensor& x, const at::Tensor* pairs, int64_t k, const char* what) {
    matrix(x, what);
    Gathered g;
    g.rows = x.size(0);
    g.x = rows_of(x, g.rows, x.size(1));
    g.P = pairs ? pairs->numel() : g.rows;
    if (pairs) {
        if (k <= 0 || k > 1 << 20) bad(std::string(what) + ": k is the number of experts of a token");
        g.pairs = vec_of<int32_t>(pairs, g.P, at::kInt);
        g.k = (int)k;
    }
    return g;
}

size_t product_bytes(const Gathered& g, const Experts& m, int op) {
    return qmoe_expert_workspace_bytes(g.P, (int)m.E, m.N, m.K, op, g.pairs != nullptr);
}

PyObject* expert_linear(const Args& a) {  // x, w, offsets, pairs, k, out_dtype, dev_status, ws
    const at::Tensor &x = a.tensor(0), &w = a.tensor(1);
    const Experts m = experts_of(w, "expert_linear");
    const Gathered g = gathered(x, a.maybe(3), a.whole(4), "expert_linear");
    if (x.size(1) != m.K) bad("the reduction lengths differ: " + shape_str(x) + " and " + shape_str(w));
    const int code = same_type(x, w, "x and w");
    const auto yt = a.dtype(5, x.scalar_type());
    const at::Tensor y = make({g.P, m.N}, yt, x);
    const int yc = code_of(yt);
    const int32_t* offsets = vec_of<int32_t>(&a.tensor(2), m.E + 1, at::kInt);
    const size_t copied = copy_of(m);
    const bool in_place = copied && qmoe_expert_linear_in_place(g.P, (int)m.E, m.N, m.K);
    const MaybeWorkspace ws(in_place ? 0 : product_bytes(g, m, 0) + copy_of(g.x, g.rows, m.K) + copied, a.maybe(7), x);
    check(qmoe_expert_linear(g.P, (int)m.E, m.N, m.K, code, g.x.p, g.x.ld, g.rows, g.pairs, g.k, m.p, m.ld, m.stride,
                             offsets, y.data_ptr(), yc, m.N, status_of(a.tensor(6)), ws.p, ws.n, stream_of(x)),
          "qmoe_expert_linear");
    return wrap(y);
}

PyObject* expert_linear_backward(const Args& a) {  // dy, x, w, offsets, pairs, k, dw_dtype, need_dx, need_dw, dev_status, ws
    const at::Tensor &dy = a.tensor(0), *x = a.maybe(1), *w = a.maybe(2), &off = a.tensor(3);
    const bool to_x = a.truth(7), to_w = a.truth(8);
    if (to_x && !w) bad("expert_linear_backward: the gradient of x takes w");
    if (to_w && !x) bad("expert_linear_backward: the gradient of w takes x");
    matrix(dy, "expert_linear_backward");
    // what is not there is of no gradient: its sizes are the others'
    Experts m;
    if (w) {
        m = experts_of(*w, "expert_linear_backward");
    } else {
        if (off.numel() < 1) bad("expert_linear_backward: expected offsets of shape [experts + 1], got " + shape_str(off));
        if (off.numel() > 1 << 20) check(QMOE_ERR_UNSUPPORTED, "expert_linear_backward");
        m.E = off.numel() - 1;
        m.N = dy.size(1);
    }
    Gathered g;
    if (x) {
        g = gathered(*x, a.maybe(4), a.whole(5), "expert_linear_backward");
        if (!w) m.K = x->size(1);
        if (x->size(1) != m.K) bad("the reduction lengths differ: " + shape_str(*x) + " and " + shape_str(*w));
    } else {
        g.P = g.rows = dy.size(0);
    }
    const Rows d = rows_of(dy, g.P, m.N);
    if (x && w) same_type(*x, *w, "x and w");
    const int code = w ? same_type(dy, *w, "dy and w") : x ? same_type(dy, *x, "dy and x") : code_of(dy.scalar_type());
    const auto wt = a.dtype(6, at::kFloat);
    const int32_t* offsets = vec_of<int32_t>(&off, m.E + 1, at::kInt);
    int32_t* const status = status_of(a.tensor(9));
    const qmoe_stream_t st = stream_of(dy);
    const size_t cd = copy_of(d, g.P, m.N), cx = to_w ? copy_of(g.x, g.rows, m.K) : 0, cw = to_x ? copy_of(m) : 0;
    const size_t need = std::max(to_x ? product_bytes(g, m, 1) + cd + cw : 0, to_w ? product_bytes(g, m, 2) + cd + cx : 0);
    const MaybeWorkspace ws(need, a.maybe(10), dy);
    at::Tensor dx, dw;
    if (to_x) {
        dx = make({g.P, m.K}, dy.scalar_type(), dy);
        check(qmoe_expert_linear_dx(g.P, (int)m.E, m.N, m.K, code, d.p, d.ld, m.p, m.ld, m.stride, offsets, dx.data_ptr(),
                                    code, m.K, status, ws.p, ws.n, st),
              "qmoe_expert_linear_dx");
    }
    if (to_w) {
        dw = make({m.E, m.N, m.K}, wt, dy);
        check(qmoe_expert_linear_dw(g.P, (int)m.E, m.N, m.K, code, d.p, d.ld, g.x.p, g.x.ld, g.rows, g.pairs, g.k, offsets,
                                    dw.data_ptr(), code_of(wt), status, ws.p, ws.n, st),
              "qmoe_expert_linear_dw");
    }
    return tuple_of({dx, dw});
}

PyObject* swiglu(const Args& a) {  // gu
    const at::Tensor& gu = a.tensor(0);
    matrix(gu, "swiglu");
    const int64_t P = gu.size(0), I = gu.size(1) / 2;
    if (gu.size(1) != 2 * I) bad("swiglu takes gate and up columns, [rows, 2 I]; got " + shape_str(gu));
    const Rows r = rows_of(gu, P, 2 * I);
    const int code = code_of(gu.scalar_type());
    const at::Tensor h = make({P, I}, gu.scalar_type(), gu);
    check(qmoe_swiglu(P, I, code, r.p, r.ld, h.data_ptr(), I, stream_of(gu)), "qmoe_swiglu");
    return wrap(h);
}

PyObject* swiglu_backward(const Args& a) {  // dh, gu, h_too
    const at::Tensor &dh = a.tensor(0), &gu = a.tensor(1);
    matrix(dh, "swiglu_backward");
    const int64_t P = dh.size(0), I = dh.size(1);
    const Rows d = rows_of(dh, P, I), r = rows_of(gu, P, 2 * I);
    const int code = code_of(gu.scalar_type());
    if (dh.scalar_type() != gu.scalar_type()) bad("dh has gu's type");
    const at::Tensor dgu = make({P, 2 * I}, gu.scalar_type(), gu);
    at::Tensor h;
    if (a.truth(2)) h = make({P, I}, gu.scalar_type(), gu);
    check(qmoe_swiglu_backward(P, I, code, d.p, d.ld, r.p, r.ld, dgu.data_ptr(), 2 * I, at_of(h), I, stream_of(gu)),
          "qmoe_swiglu_backward");
    return tuple_of({dgu, h});
}

struct Slots {
    int64_t T, k;
    const int32_t* p;
};
Slots slots_of(const at::Tensor& t, const char* what) {
    if (t.dim() != 2) bad(std::string(what) + ": expected pair_slot of shape [tokens, k], got " + shape_str(t));
    if (t.size(1) > 1 << 20) check(QMOE_ERR_UNSUPPORTED, what);
    return {t.size(0), t.size(1), vec_of<int32_t>(&t, t.numel(), at::kInt)};
}

PyObject* combine(const Args& a) {  // y, w, pair_slot
    const at::Tensor& y = a.tensor(0);
    matrix(y, "combine");
    const Slots s = slots_of(a.tensor(2), "combine");
    const int64_t P = y.size(0), H = y.size(1);
    const Rows r = rows_of(y, P, H);
    const int code = code_of(y.scalar_type());
    const float* w = floats(a.maybe(1), s.T * s.k);
    const at::Tensor out = make({s.T, H}, y.scalar_type(), y);
    check(qmoe_weighted_sum(s.T, (int)s.k, P, H, code, r.p, r.ld, w, s.p, out.data_ptr(), H, stream_of(y)), "qmoe_weighted_sum");
    return wrap(out);
}

PyObject* combine_backward(const Args& a) {  // dout, y, w, pair_slot, offsets
    const at::Tensor &dout = a.tensor(0), &y = a.tensor(1), *w = a.maybe(2), &offsets = a.tensor(4);
    matrix(y, "combine_backward");
    const Slots s = slots_of(a.tensor(3), "combine_backward");
    const int64_t P = y.size(0), H = y.size(1), E = offsets.numel() - 1;
    const Rows d = rows_of(dout, s.T, H), r = rows_of(y, P, H);
    const int code = code_of(y.scalar_type());
    if (dout.scalar_type() != y.scalar_type()) bad("dout has y's type");
    if (E < 0) bad("combine_backward: expected offsets of shape [experts + 1], got " + shape_str(offsets));
    const int32_t* routed = vec_of<int32_t>(&offsets, E + 1, at::kInt) + E;
    const float* wp = floats(w, s.T * s.k);
    at::Tensor dy = make({P, H}, y.scalar_type(), y), dw;
    if (w) dw = make({s.T, s.k}, at::kFloat, y);
    if (P == 0 && w) dw.zero_();
    else
        check(qmoe_weighted_sum_backward(s.T, (int)s.k, P, H, code, d.p, d.ld, w ? r.p : nullptr, r.ld, wp, s.p, routed,
                                         dy.data_ptr(), H, f32_of(dw), stream_of(y)),
              "qmoe_weighted_sum_backward");
    return tuple_of({dy, dw});
}

// ------------------------------------------------------------------ 4-bit products

struct Codes4 {
    int64_t E = 1, N, K;
    int format, group;
    const uint8_t* w;
    const void* s;
};
Codes4 codes4_of(const at::Tensor& q, const at::Tensor& s, bool experts, const char* what) {
    const int64_t d = experts ? 3 : 2;
    if (q.dim() != d || s.dim() != d || q.scalar_type() != at::kByte)
        bad(std::string(what) + ": expected uint8 codes and scales of " + (experts ? "[experts, outputs, ...]" : "[outputs, ...]") +
            ", got " + shape_str(q) + " and " + shape_str(s));
    Codes4 c;
    c.E = experts ? q.size(0) : 1;
    c.N = q.size(d - 2);
    c.K = q.size(d - 1) * 2;
    const int64_t groups = s.size(d - 1);
    if ((experts && s.size(0) != c.E) || s.size(d - 2) != c.N || groups <= 0 || c.K % groups || c.K / groups > 1 << 20)
        bad(std::string(what) + ": codes and scales do not go together: " + shape_str(q) + " and " + shape_str(s));
    c.group = (int)(c.K / groups);
    if (s.scalar_type() == at::kHalf) c.format = QMOE_W4_INT4;
    else if (s.scalar_type() == at::kByte) c.format = QMOE_W4_E2M1;
    else bad(std::string(what) + ": scales are float16 (int4 codes) or uint8 (E2M1 codes), got " + shape_str(s));
    if (c.E > 1 << 20) check(QMOE_ERR_UNSUPPORTED, what);
    on_device(q);
    on_device(s);
    if (!q.is_contiguous() || !s.is_contiguous()) refuse(qmoe_error, "qmoe kernels take contiguous tensors");
    c.w = static_cast<const uint8_t*>(q.data_ptr());
    c.s = s.data_ptr();
    return c;
}

PyObject* w4_linear(const Args& a) {  // x, w_q, w_s, ids, out_dtype, dev_status, ws
    const at::Tensor &x = a.tensor(0), *ids = a.maybe(3);
    matrix(x, "w4_linear");
    const Codes4 c = codes4_of(a.tensor(1), a.tensor(2), ids != nullptr, "w4_linear");
    const int64_t T = x.size(0), k = ids ? (ids->dim() == 2 ? ids->size(1) : -1) : 1;
    if (ids && (k <= 0 || k > 65535 || ids->size(0) != T)) bad("w4_linear: expected ids of shape [tokens, k], got " + shape_str(*ids));
    if (x.size(1) != c.K) bad("the reduction lengths differ: " + shape_str(x) + " and " + shape_str(a.tensor(1)));
    const Rows r = rows_of(x, T, c.K);
    const int code = code_of(x.scalar_type());
    if (code == QMOE_F32) bad("w4_linear: x is of bfloat16 or float16");
    const auto yt = a.dtype(4, x.scalar_type());
    const int yc = code_of(yt);
    const at::Tensor y = make({T * k, c.N}, yt, x);
    const MaybeWorkspace ws(ids ? 0 : qmoe_w4_workspace_bytes(T, c.N, c.K, 0), a.maybe(6), x);
    check(qmoe_w4_linear(T, (int)k, (int)c.E, c.N, c.K, c.format, c.group, code, r.p, r.ld, c.w, c.s,
                         vec_of<int32_t>(ids, T * k, at::kInt), y.data_ptr(), yc, c.N, status_of(a.tensor(5)), ws.p, ws.n,
                         stream_of(x)),
          "qmoe_w4_linear");
    return wrap(y);
}

PyObject* w4_linear_backward(const Args& a) {  // dy, w_q, w_s, dev_status, ws
    const at::Tensor& dy = a.tensor(0);
    matrix(dy, "w4_linear_backward");
    const Codes4 c = codes4_of(a.tensor(1), a.tensor(2), false, "w4_linear_backward");
    const int64_t T = dy.size(0);
    const Rows r = rows_of(dy, T, c.N);
    const int code = code_of(dy.scalar_type());
    if (code == QMOE_F32) bad("w4_linear_backward: dy is of bfloat16 or float16");
    const at::Tensor dx = make({T, c.K}, dy.scalar_type(), dy);
    const MaybeWorkspace ws(qmoe_w4_workspace_bytes(T, c.N, c.K, 1), a.maybe(4), dy);
    check(qmoe_w4_linear_dx(T, c.N, c.K, c.format, c.group, code, r.p, r.ld, c.w, c.s, dx.data_ptr(), code, c.K,
                            status_of(a.tensor(3)), ws.p, ws.n, stream_of(dy)),
          "qmoe_w4_linear_dx");
    return wrap(dx);
}

// ------------------------------------------------------------------ module

template <PyObject* (*F)(const Args&), int N>
PyObject* entry(PyObject* self, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        const Args a(v, n, N, PyModule_GetName(self));
        const std::optional<at::Device> device = a.device();
        c10::cuda::OptionalCUDAGuard guard;
        if (device && device->index() != c10::cuda::current_device()) guard.set_device(*device);
        return F(a);
    } catch (const PythonError&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* init(PyObject*, PyObject* error) {
    Py_XDECREF(qmoe_error);
    Py_INCREF(error);
    qmoe_error = error;
    Py_RETURN_NONE;
}

#define ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"init", init, METH_O, "init(error): the exception class for what the library refuses"},
    ENTRY(norm_pre, 4),
    ENTRY(norm_pre_backward, 6),
    ENTRY(norm_post, 7),
    ENTRY(norm_post_backward, 11),
    ENTRY(route_topk, 8),
    ENTRY(route_topk_backward, 10),
    ENTRY(fp8_quant_rows, 1),
    ENTRY(fp8_quant_cols, 2),
    ENTRY(fp8_quant_blocks, 2),
    ENTRY(fp8_matmul, 6),
    ENTRY(fp8_linear, 6),
    ENTRY(fp8_linear_backward, 5),
    ENTRY(expert_linear, 8),
    ENTRY(expert_linear_backward, 11),
    ENTRY(swiglu, 1),
    ENTRY(swiglu_backward, 3),
    ENTRY(combine, 3),
    ENTRY(combine_backward, 5),
    ENTRY(w4_linear, 7),
    ENTRY(w4_linear_backward, 5),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
