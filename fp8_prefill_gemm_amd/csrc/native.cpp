// Native half of the binding's MXFP4 and cache calls: argument checks, output
// allocation, the current stream and the call into librz_fp8.so, for torch
// tensors.  On small batches a kernel takes 3 to 5 us; a call with these steps
// in Python took 8.6 us of the host's time, 4.3 to 4.8 so, of it 3.2 to 3.7
// the C call.
// The Python functions in __init__.py carry the names, defaults and
// documentation.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <sstream>
#include <string>

#include "../../include/rz_fp8.h"

namespace {

using at::Tensor;
using Shape = std::initializer_list<int64_t>;

PyObject* g_error = nullptr;  // RzError

struct Failed {  // a call's negative status
    int status;
};

[[noreturn]] void refuse(const std::string& msg) {
    TORCH_CHECK_VALUE(false, msg);
    __builtin_unreachable();
}

std::string shape_text(c10::IntArrayRef s) {
    std::ostringstream o;
    o << s;
    return o.str();
}

[[noreturn]] void refuse_tensor(const Tensor& t, const char* what, at::ScalarType dtype, c10::IntArrayRef shape) {
    std::ostringstream o;
    o << what << ": expected a contiguous " << dtype << " tensor of shape " << shape << ", got " << t.scalar_type() << " "
      << t.sizes() << " with strides " << t.strides();
    refuse(o.str());
}

void in_range(int64_t v, const char* what, int64_t lo, int64_t hi) {
    if (v < lo || v > hi) {
        std::ostringstream o;
        o << what << "=" << v << ": expected " << lo << " to " << hi;
        refuse(o.str());
    }
}

// Every size here goes to the library as a uint32.
constexpr int64_t kMaxSize = 0xFFFFFFFFll;

// Size `axis` of t times `per`, in that range.
int64_t size_of(const Tensor& t, int64_t axis, const char* what, int64_t per = 1) {
    const int64_t v = t.size(axis);
    in_range(v > kMaxSize ? v : v * per, what, 0, kMaxSize);
    return v * per;
}

// The arguments of one call, in order.
struct Args {
    PyObject* const* a;
    Py_ssize_t n;

    const Tensor& tensor(Py_ssize_t i, const char* what) const {
        TORCH_CHECK_TYPE(THPVariable_Check(a[i]), what, ": expected a tensor, got ", Py_TYPE(a[i])->tp_name);
        return THPVariable_Unpack(a[i]);
    }
    bool none(Py_ssize_t i) const { return a[i] == Py_None; }
    // a whole number in [lo, hi]
    int64_t number(Py_ssize_t i, const char* what, int64_t lo = 0, int64_t hi = kMaxSize) const {
        PyObject* x = PyNumber_Index(a[i]);
        if (!x) throw python_error();
        const int64_t v = PyLong_AsLongLong(x);
        Py_DECREF(x);
        if (v == -1 && PyErr_Occurred()) throw python_error();
        in_range(v, what, lo, hi);
        return v;
    }
    // a floating-point number, as the library takes it
    float real(Py_ssize_t i) const {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) throw python_error();
        return (float)v;
    }
};

void need(const Tensor& t, const char* what, at::ScalarType dtype, c10::IntArrayRef shape) {
    if (t.scalar_type() != dtype || t.sizes() != shape || !t.is_contiguous() || t.layout() != at::kStrided)
        refuse_tensor(t, what, dtype, shape);
}

// One GPU for every tensor of a call, checked after their shapes.
struct Device {
    const Tensor& first;
    explicit Device(const Tensor& t) : first(t) {
        if (!t.is_cuda()) refuse("rz_fp8 works on device (cuda/hip) tensors only");
    }
    const Device& same(std::initializer_list<const Tensor*> ts) const {
        for (const Tensor* t : ts)
            if (t->device() != first.device()) {
                std::ostringstream o;
                o << "rz_fp8: tensors on " << t->device() << " and " << first.device() << ": one device expected";
                refuse(o.str());
            }
        return *this;
    }
};

// The stream of a call, argument i: a handle, or None for torch's current
// stream on the call's device.  For the object's life it is torch's current
// one there, so that the outputs made below are the allocator's blocks for it.
struct OnStream {
    const Device& dev;
    const c10::hip::HIPStream before;
    void* handle;
    OnStream(const Args& A, Py_ssize_t i, const Device& d)
        : dev(d), before(c10::hip::getCurrentHIPStream(d.first.get_device())), handle(before.stream()) {
        if (A.none(i)) return;
        handle = PyLong_AsVoidPtr(A.a[i]);
        if (PyErr_Occurred()) throw python_error();
        if (other()) c10::hip::setCurrentHIPStream(c10::hip::getStreamFromExternal(static_cast<hipStream_t>(handle), d.first.get_device()));
    }
    ~OnStream() {
        if (other()) c10::hip::setCurrentHIPStream(before);
    }
    bool other() const { return handle != before.stream(); }
    OnStream(const OnStream&) = delete;
};

// The output argument i, checked, or a new tensor.
Tensor output(const Args& A, Py_ssize_t i, const char* what, at::ScalarType dtype, c10::IntArrayRef shape, const OnStream& on) {
    if (A.none(i)) return at::empty(shape, on.dev.first.options().dtype(dtype).layout(at::kStrided).requires_grad(false));
    const Tensor& t = A.tensor(i, what);
    need(t, what, dtype, shape);
    on.dev.same({&t});
    return t;
}

// Calls f(stream) with the call's device current.
template <typename F>
void call(const OnStream& on, F&& f) {
    const int index = on.dev.first.get_device();
    int current = index;
    const bool other = hipGetDevice(&current) == hipSuccess && current != index;
    if (other) (void)hipSetDevice(index);
    const int status = f(on.handle);
    if (other) (void)hipSetDevice(current);
    if (status != RZ_OK) throw Failed{status};
}

template <typename T = uint8_t>
T* ptr(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

// An MXFP4 tensor argument pair (codes, scales) of `rows` rows.
struct Mx {
    const Tensor &codes, &scales;
    int64_t k;
    Mx(const Args& A, Py_ssize_t i, int64_t rows, const char* what)
        : codes(A.tensor(i, what)), scales(A.tensor(i + 1, what)), k(codes.dim() == 3 ? size_of(codes, 1, "k", 64) : 0) {
        const int64_t g = (rows + 31) / 32;
        need(codes, what, at::kByte, Shape{g, k / 64, 1024});
        need(scales, what, at::kByte, Shape{g, k / 256, 256});
    }
};

void same_k(const Mx& a, const Mx& b, const char* what) {
    if (a.k != b.k) refuse(std::string(what) + ": operands have k=" + std::to_string(a.k) + " and k=" + std::to_string(b.k));
}

struct MxOut {
    Tensor codes, scales;
    MxOut(const Args& A, Py_ssize_t i, int64_t rows, int64_t k, const char* what, const OnStream& on) {
        const int64_t g = (rows + 31) / 32;
        codes = output(A, i, what, at::kByte, Shape{g, k / 64, 1024}, on);
        scales = output(A, i + 1, what, at::kByte, Shape{g, k / 256, 256}, on);
    }
};

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

PyObject* wrap2(const Tensor& a, const Tensor& b) {
    PyObject *x = wrap(a), *y = wrap(b);
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

at::ScalarType dtype_of(int64_t id) { return id == RZ_F32 ? at::kFloat : id == RZ_F16 ? at::kHalf : at::kBFloat16; }

// (x, codes, scales, stream)
PyObject* mxfp4_quant(const Args& A) {
    const Tensor& x = A.tensor(0, "x");
    if (x.dim() != 2) refuse("x: expected 2 dimensions, got " + shape_text(x.sizes()));
    const int64_t m = size_of(x, 0, "m"), k = size_of(x, 1, "k");
    need(x, "x", at::kFloat, Shape{m, k});
    const Device dev(x);
    const OnStream on(A, 3, dev);
    MxOut o(A, 1, m, k, "output", on);
    call(on, [&](void* st) { return rz_mxfp4_quant(ptr<float>(x), m, k, ptr(o.codes), ptr(o.scales), st); });
    return wrap2(o.codes, o.scales);
}

// (qtype, blocks, n, k, codes, scales, stream)
PyObject* mxfp4_pack_weight(const Args& A) {
    const int64_t qtype = A.number(0, "qtype"), n = A.number(2, "n"), k = A.number(3, "k");
    const Tensor& b = A.tensor(1, "blocks");
    need(b, "blocks", at::kByte, b.sizes());
    const int64_t bytes = (int64_t)rz_weight_bytes((int)qtype, n, k);
    if (b.numel() < bytes) refuse("blocks: " + std::to_string(b.numel()) + " bytes, " + std::to_string(bytes) + " needed");
    const Device dev(b);
    const OnStream on(A, 6, dev);
    MxOut o(A, 4, n, k, "output", on);
    call(on, [&](void* st) { return rz_mxfp4_pack_weight((int)qtype, ptr(b), n, k, ptr(o.codes), ptr(o.scales), st); });
    return wrap2(o.codes, o.scales);
}

// (codes, scales, rows, out, dtype id, stream)
PyObject* mxfp4_dequant(const Args& A) {
    const int64_t rows = A.number(2, "rows"), id = A.number(4, "dtype", 0, 2);
    const Mx c(A, 0, rows, "input");
    const Device dev(c.codes);
    dev.same({&c.scales});
    const OnStream on(A, 5, dev);
    const Tensor out = output(A, 3, "out", dtype_of(id), Shape{rows, c.k}, on);
    call(on, [&](void* st) { return rz_mxfp4_dequant(ptr(c.codes), ptr(c.scales), rows, c.k, (int)id, ptr<void>(out), st); });
    return wrap(out);
}

// (a_codes, a_scales, m, w_codes, w_scales, n, y, stream)
PyObject* mxfp4_gemm(const Args& A) {
    const int64_t m = A.number(2, "m"), n = A.number(5, "n");
    const Mx a(A, 0, m, "a"), w(A, 3, n, "w");
    same_k(a, w, "a and w");
    const Device dev(a.codes);
    dev.same({&a.scales, &w.codes, &w.scales});
    const OnStream on(A, 7, dev);
    const Tensor y = output(A, 6, "y", at::kFloat, Shape{m, n}, on);
    call(on, [&](void* st) {
        return rz_mxfp4_gemm(ptr(a.codes), ptr(a.scales), m, ptr(w.codes), ptr(w.scales), n, a.k, ptr<float>(y), st);
    });
    return wrap(y);
}

// (a_codes, a_scales, m, gate codes, gate scales, up codes, up scales, n, h, stream)
PyObject* mxfp4_gated(const Args& A) {
    const int64_t m = A.number(2, "m"), n = A.number(7, "n");
    const Mx a(A, 0, m, "a"), g(A, 3, n, "gate"), u(A, 5, n, "up");
    same_k(a, g, "a and gate");
    same_k(a, u, "a and up");
    const Device dev(a.codes);
    dev.same({&a.scales, &g.codes, &g.scales, &u.codes, &u.scales});
    const OnStream on(A, 9, dev);
    const Tensor h = output(A, 8, "h", at::kFloat, Shape{m, n}, on);
    call(on, [&](void* st) {
        return rz_mxfp4_gated(ptr(a.codes), ptr(a.scales), m, ptr(g.codes), ptr(g.scales), ptr(u.codes), ptr(u.scales), n, a.k,
                              ptr<float>(h), st);
    });
    return wrap(h);
}

// (a_codes, a_scales, m, gate codes, gate scales, up codes, up scales, n, h_codes, h_scales, stream)
PyObject* mxfp4_gated_quant(const Args& A) {
    const int64_t m = A.number(2, "m"), n = A.number(7, "n");
    const Mx a(A, 0, m, "a"), g(A, 3, n, "gate"), u(A, 5, n, "up");
    same_k(a, g, "a and gate");
    same_k(a, u, "a and up");
    const Device dev(a.codes);
    dev.same({&a.scales, &g.codes, &g.scales, &u.codes, &u.scales});
    const OnStream on(A, 10, dev);
    MxOut o(A, 8, m, n, "h", on);
    call(on, [&](void* st) {
        return rz_mxfp4_gated_quant(ptr(a.codes), ptr(a.scales), m, ptr(g.codes), ptr(g.scales), ptr(u.codes), ptr(u.scales), n,
                                    a.k, ptr(o.codes), ptr(o.scales), st);
    });
    return wrap2(o.codes, o.scales);
}

// x fp32 [m][k] of a GEMV.
int64_t gemv_rows(const Tensor& x, int64_t k) {
    const int64_t m = x.dim() == 2 ? size_of(x, 0, "m") : 0;
    need(x, "x", at::kFloat, Shape{m, k});
    return m;
}

// (w_codes, w_scales, n, x, y, stream)
PyObject* mxfp4_gemv(const Args& A) {
    const int64_t n = A.number(2, "n");
    const Mx w(A, 0, n, "w");
    const Tensor& x = A.tensor(3, "x");
    const int64_t m = gemv_rows(x, w.k);
    const Device dev(x);
    dev.same({&w.codes, &w.scales});
    const OnStream on(A, 5, dev);
    const Tensor y = output(A, 4, "y", at::kFloat, Shape{m, n}, on);
    call(on, [&](void* st) { return rz_mxfp4_gemv(ptr(w.codes), ptr(w.scales), n, w.k, ptr<float>(x), m, ptr<float>(y), st); });
    return wrap(y);
}

// (gate codes, gate scales, up codes, up scales, n, x, h, stream)
PyObject* mxfp4_gated_gemv(const Args& A) {
    const int64_t n = A.number(4, "n");
    const Mx g(A, 0, n, "gate"), u(A, 2, n, "up");
    same_k(g, u, "gate and up");
    const Tensor& x = A.tensor(5, "x");
    const int64_t m = gemv_rows(x, g.k);
    const Device dev(x);
    dev.same({&g.codes, &g.scales, &u.codes, &u.scales});
    const OnStream on(A, 7, dev);
    const Tensor h = output(A, 6, "h", at::kFloat, Shape{m, n}, on);
    call(on, [&](void* st) {
        return rz_mxfp4_gated_gemv(ptr(g.codes), ptr(g.scales), ptr(u.codes), ptr(u.scales), n, g.k, ptr<float>(x), m,
                                   ptr<float>(h), st);
    });
    return wrap(h);
}

// One tensor pair of a cache (its keys): format argument i, codes and scales from argument j on.
struct KeyRows {
    int64_t fmt, slots, heads, dim;
    const Tensor &kc, &ks;
    KeyRows(const Args& A, Py_ssize_t i, Py_ssize_t j)
        : fmt(A.number(i, "fmt", 0, 1)), kc(A.tensor(j, "k_codes")), ks(A.tensor(j + 1, "k_scales")) {
        if (kc.dim() != 3) refuse("k_codes: expected 3 dimensions, got " + shape_text(kc.sizes()));
        slots = kc.size(0);
        heads = size_of(kc, 1, "heads");
        dim = size_of(kc, 2, "dim", fmt == RZ_KV_E4M3 ? 1 : 2);
        need(kc, "k_codes", at::kByte, kc.sizes());
    }
    void scales_of(const Tensor& s, const char* what) const {
        if (fmt == RZ_KV_E4M3)
            need(s, what, at::kFloat, Shape{slots, heads});
        else
            need(s, what, at::kByte, Shape{slots, heads, kc.size(2) / 16});
    }
};

// A whole cache: k_codes, k_scales, v_codes, v_scales from argument j on.
struct Cache : KeyRows {
    const Tensor &vc, &vs;
    Cache(const Args& A, Py_ssize_t i, Py_ssize_t j) : KeyRows(A, i, j), vc(A.tensor(j + 2, "v_codes")), vs(A.tensor(j + 3, "v_scales")) {
        need(vc, "v_codes", at::kByte, Shape{slots, heads, kc.size(2)});
        scales_of(ks, "k_scales");
        scales_of(vs, "v_scales");
    }
};

// The token stride of t, fp32 [tokens][heads][dim] with contiguous tokens.
int64_t token_stride(const Tensor& t, const char* what, int64_t tokens, int64_t heads, int64_t dim) {
    const int64_t shape[3] = {tokens, heads, dim};
    if (t.scalar_type() != at::kFloat || t.layout() != at::kStrided || t.sizes() != c10::IntArrayRef(shape) ||
        (tokens > 0 && ((dim > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != dim))) ||
        (tokens > 1 && t.stride(0) < heads * dim))
        refuse_tensor(t, what, at::kFloat, shape);
    return tokens > 1 ? t.stride(0) : heads * dim;  // free where there is one token
}

// (fmt, k, v, slots, k_codes, k_scales, v_codes, v_scales, stream)
PyObject* kv_cache_write(const Args& A) {
    const Cache c(A, 0, 4);
    const Tensor &k = A.tensor(1, "k"), &v = A.tensor(2, "v"), &slots = A.tensor(3, "slots");
    const int64_t tokens = k.dim() == 3 ? size_of(k, 0, "tokens") : 0;
    const int64_t ks = token_stride(k, "k", tokens, c.heads, c.dim), vs = token_stride(v, "v", tokens, c.heads, c.dim);
    need(slots, "slots", at::kLong, Shape{tokens});
    const Device dev(k);
    dev.same({&v, &slots, &c.kc, &c.ks, &c.vc, &c.vs});
    const OnStream on(A, 8, dev);
    call(on, [&](void* st) {
        return rz_kv_cache_write((int)c.fmt, ptr<float>(k), ptr<float>(v), tokens, c.heads, c.dim, ks, vs, ptr<int64_t>(slots),
                                 c.slots, ptr(c.kc), ptr<void>(c.ks), ptr(c.vc), ptr<void>(c.vs), st);
    });
    Py_RETURN_NONE;
}

// (fmt, k_codes, k_scales, v_codes, v_scales, page_len, page_table, offsets, rows, k_out, v_out, dtype id, stream)
PyObject* kv_cache_read(const Args& A) {
    const Cache c(A, 0, 1);
    const int64_t page_len = A.number(5, "page_len", 1), rows = A.number(8, "rows"), id = A.number(11, "dtype", 0, 2);
    const Tensor &table = A.tensor(6, "page_table"), &offsets = A.tensor(7, "offsets");
    if (table.dim() != 2) refuse("page_table: expected 2 dimensions, got " + shape_text(table.sizes()));
    const int64_t seqs = size_of(table, 0, "sequences"), pages = size_of(table, 1, "pages");
    need(table, "page_table", at::kInt, Shape{seqs, pages});
    need(offsets, "offsets", at::kInt, Shape{seqs + 1});
    const Device dev(c.kc);
    dev.same({&c.ks, &c.vc, &c.vs, &table, &offsets});
    const OnStream on(A, 12, dev);
    const Tensor k = output(A, 9, "k_out", dtype_of(id), Shape{rows, c.heads, c.dim}, on);
    const Tensor v = output(A, 10, "v_out", dtype_of(id), Shape{rows, c.heads, c.dim}, on);
    call(on, [&](void* st) {
        return rz_kv_cache_read((int)c.fmt, ptr(c.kc), ptr<void>(c.ks), ptr(c.vc), ptr<void>(c.vs), c.slots, c.heads, c.dim,
                                page_len, ptr<int32_t>(table), seqs, pages, ptr<int32_t>(offsets), rows, (int)id, ptr<void>(k),
                                ptr<void>(v), st);
    });
    return wrap2(k, v);
}

// A new workspace of the call's stream (null where it is empty).
Tensor workspace(size_t bytes, const OnStream& on) {
    if (bytes == 0) return Tensor();
    return at::empty({(int64_t)bytes}, on.dev.first.options().dtype(at::kByte).layout(at::kStrided).requires_grad(false));
}
void* at_or_null(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// (lens, keep, offsets, tokens, page_len, page_table, free_pages, free_count, lens_out, count_out, slots, stream)
PyObject* kv_plan(const Args& A) {
    const Tensor &lens = A.tensor(0, "lens"), &offsets = A.tensor(2, "offsets"), &table = A.tensor(5, "page_table"),
                 &free = A.tensor(6, "free_pages"), &count = A.tensor(7, "free_count");
    const int64_t tokens = A.number(3, "tokens"), page_len = A.number(4, "page_len", 1);
    if (table.dim() != 2) refuse("page_table: expected 2 dimensions, got " + shape_text(table.sizes()));
    const int64_t seqs = size_of(table, 0, "sequences"), max_pages = size_of(table, 1, "pages");
    if (free.dim() != 1) refuse("free_pages: expected 1 dimension, got " + shape_text(free.sizes()));
    const int64_t pages = size_of(free, 0, "num_pages");
    need(lens, "lens", at::kInt, Shape{seqs});
    need(offsets, "offsets", at::kInt, Shape{seqs + 1});
    need(table, "page_table", at::kInt, Shape{seqs, max_pages});
    need(free, "free_pages", at::kInt, Shape{pages});
    need(count, "free_count", at::kInt, Shape{1});
    const Tensor& keep = A.none(1) ? lens : A.tensor(1, "keep");  // all of them by default
    need(keep, "keep", at::kInt, Shape{seqs});
    const Device dev(lens);
    dev.same({&keep, &offsets, &table, &free, &count});
    const OnStream on(A, 11, dev);
    const Tensor then = output(A, 8, "lens_out", at::kInt, Shape{seqs}, on), left = output(A, 9, "count_out", at::kInt, Shape{1}, on),
                 slots = output(A, 10, "slots", at::kLong, Shape{tokens}, on);
    const Tensor ws = workspace(rz_kv_plan_workspace_bytes(seqs, tokens), on);
    call(on, [&](void* st) {
        return rz_kv_plan(ptr<int32_t>(lens), ptr<int32_t>(keep), ptr<int32_t>(offsets), seqs, tokens, page_len, ptr<int32_t>(table), max_pages,
                          ptr<int32_t>(free), pages, ptr<int32_t>(count), ptr<int32_t>(then), ptr<int32_t>(left),
                          ptr<int64_t>(slots), at_or_null(ws), st);
    });
    PyObject *x = wrap(slots), *y = wrap(then), *z = wrap(left);
    PyObject* r = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return r;
}

// The queries, page table and lengths of a serving call.
struct Queries {
    const Tensor &q, &table, &lens;
    int64_t seqs, q_heads, max_pages, stride;
    Queries(const Args& A, Py_ssize_t iq, Py_ssize_t it, Py_ssize_t il, int64_t dim)
        : q(A.tensor(iq, "q")), table(A.tensor(it, "page_table")), lens(A.tensor(il, "lens")) {
        if (table.dim() != 2) refuse("page_table: expected 2 dimensions, got " + shape_text(table.sizes()));
        seqs = size_of(table, 0, "sequences");
        max_pages = size_of(table, 1, "pages");
        q_heads = q.dim() == 3 ? size_of(q, 1, "q_heads") : 0;
        stride = token_stride(q, "q", seqs, q_heads, dim);
        need(table, "page_table", at::kInt, Shape{seqs, max_pages});
        need(lens, "lens", at::kInt, Shape{seqs});
    }
};

// (fmt, q, k_codes, k_scales, v_codes, v_scales, page_len, page_table, lens, scale, pages, out, dtype id, lse, stream)
PyObject* kv_attention(const Args& A) {
    const Cache c(A, 0, 2);
    const int64_t page_len = A.number(6, "page_len", 1), id = A.number(12, "dtype", 0, 2);
    const Queries s(A, 1, 7, 8, c.dim);
    const float scale = A.real(9);
    const Tensor* chosen = nullptr;
    int64_t budget = 0;
    if (!A.none(10)) {
        chosen = &A.tensor(10, "pages");
        if (chosen->dim() != 3) refuse("pages: expected 3 dimensions, got " + shape_text(chosen->sizes()));
        budget = size_of(*chosen, 2, "budget");
        need(*chosen, "pages", at::kInt, Shape{s.seqs, c.heads, budget});
    }
    const Tensor* lse = nullptr;
    if (!A.none(13)) {
        lse = &A.tensor(13, "lse");
        need(*lse, "lse", at::kFloat, Shape{s.seqs, s.q_heads});
    }
    const Device dev(s.q);
    dev.same({&c.kc, &c.ks, &c.vc, &c.vs, &s.table, &s.lens});
    if (chosen) dev.same({chosen});
    if (lse) dev.same({lse});
    // an empty choice has no memory, which the library would take for no choice
    const int32_t* pages = !chosen ? nullptr : budget ? ptr<int32_t>(*chosen) : ptr<int32_t>(s.lens);
    const OnStream on(A, 14, dev);
    const Tensor out = output(A, 11, "out", dtype_of(id), Shape{s.seqs, s.q_heads, c.dim}, on);
    const Tensor ws = workspace(rz_kv_attention_workspace_bytes(s.seqs, s.q_heads, c.heads, c.dim), on);
    call(on, [&](void* st) {
        return rz_kv_attention((int)c.fmt, ptr<float>(s.q), s.q_heads, s.stride, ptr(c.kc), ptr<void>(c.ks), ptr(c.vc),
                               ptr<void>(c.vs), c.slots, c.heads, c.dim, page_len, ptr<int32_t>(s.table), s.seqs, s.max_pages,
                               ptr<int32_t>(s.lens), pages, budget, scale, (int)id, ptr<void>(out), lse ? ptr<float>(*lse) : nullptr,
                               at_or_null(ws), st);
    });
    return wrap(out);
}

// int8 [num_pages][heads][2][dim] and fp32 [num_pages][heads]
struct PageBounds {
    const Tensor &codes, &scales;
    int64_t pages, heads, dim;
    PageBounds(const Args& A, Py_ssize_t i) : codes(A.tensor(i, "bounds")), scales(A.tensor(i + 1, "bound_scales")) {
        if (codes.dim() != 4) refuse("bounds: expected 4 dimensions, got " + shape_text(codes.sizes()));
        pages = size_of(codes, 0, "num_pages");
        heads = size_of(codes, 1, "heads");
        dim = size_of(codes, 3, "dim");
        need(codes, "bounds", at::kChar, Shape{pages, heads, 2, dim});
        need(scales, "bound_scales", at::kFloat, Shape{pages, heads});
    }
};

// (fmt, k_codes, k_scales, slots, page_len, bounds, bound_scales, stream)
PyObject* kv_bounds(const Args& A) {
    const KeyRows c(A, 0, 1);
    c.scales_of(c.ks, "k_scales");
    const Tensor& slots = A.tensor(3, "slots");
    const int64_t page_len = A.number(4, "page_len", 1);
    const PageBounds b(A, 5);
    if (slots.dim() != 1) refuse("slots: expected 1 dimension, got " + shape_text(slots.sizes()));
    const int64_t tokens = size_of(slots, 0, "tokens");
    need(slots, "slots", at::kLong, Shape{tokens});
    if (b.pages != c.slots / page_len || b.heads != c.heads || b.dim != c.dim)
        refuse_tensor(b.codes, "bounds", at::kChar, {c.slots / page_len, c.heads, 2, c.dim});
    const Device dev(c.kc);
    dev.same({&c.ks, &slots, &b.codes, &b.scales});
    const OnStream on(A, 7, dev);
    call(on, [&](void* st) {
        return rz_kv_bounds((int)c.fmt, ptr(c.kc), ptr<void>(c.ks), c.slots, c.heads, c.dim, page_len, ptr<int64_t>(slots), tokens,
                            ptr<int8_t>(b.codes), ptr<float>(b.scales), st);
    });
    Py_RETURN_NONE;
}

// (q, bounds, bound_scales, page_len, page_table, lens, budget, pages, stream)
PyObject* kv_select(const Args& A) {
    const PageBounds b(A, 1);
    const int64_t page_len = A.number(3, "page_len", 1), budget = A.number(6, "budget", 1);
    const Queries s(A, 0, 4, 5, b.dim);
    const Device dev(s.q);
    dev.same({&b.codes, &b.scales, &s.table, &s.lens});
    const OnStream on(A, 8, dev);
    const Tensor pages = output(A, 7, "pages", at::kInt, Shape{s.seqs, b.heads, budget}, on);
    const Tensor ws = workspace(rz_kv_select_workspace_bytes(s.seqs, b.heads, s.max_pages), on);
    call(on, [&](void* st) {
        return rz_kv_select(ptr<float>(s.q), s.q_heads, s.stride, ptr<int8_t>(b.codes), ptr<float>(b.scales), b.pages, b.heads, b.dim,
                            page_len, ptr<int32_t>(s.table), s.seqs, s.max_pages, ptr<int32_t>(s.lens), budget,
                            ptr<int32_t>(pages), at_or_null(ws), st);
    });
    return wrap(pages);
}

// One Python-callable function of N arguments.
template <PyObject* (*F)(const Args&), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(Args{args, n});
    } catch (const Failed& f) {
        PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", f.status, rz_last_error_string()) : nullptr;
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        } else if (!PyErr_Occurred()) {
            PyErr_SetString(PyExc_RuntimeError, rz_last_error_string());
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

#define RZ_ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    RZ_ENTRY(mxfp4_quant, 4),      RZ_ENTRY(mxfp4_pack_weight, 7), RZ_ENTRY(mxfp4_dequant, 6),
    RZ_ENTRY(mxfp4_gemm, 8),       RZ_ENTRY(mxfp4_gated, 10),      RZ_ENTRY(mxfp4_gated_quant, 11),
    RZ_ENTRY(mxfp4_gemv, 6),       RZ_ENTRY(mxfp4_gated_gemv, 8),  RZ_ENTRY(kv_cache_write, 9),
    RZ_ENTRY(kv_cache_read, 13),   RZ_ENTRY(kv_plan, 12),          RZ_ENTRY(kv_attention, 15),
    RZ_ENTRY(kv_bounds, 8),        RZ_ENTRY(kv_select, 9),         {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
#undef RZ_ENTRY

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rz_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__rz_native(void) { return PyModule_Create(&module); }
