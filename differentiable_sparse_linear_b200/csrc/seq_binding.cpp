// The torch side of the sequence operators (include/sla.h, "sequence operators"): argument checks, output
// and scratch allocation and the call, in one native function each.  These calls take microseconds on the
// device, so a decoding loop pays for every step of the host's; the checks in Python cost more than the kernels.
//
// Every function takes its arguments by position (None where absent) and returns tensors.  A wrong argument
// raises ValueError before any device work, a failing library call sla's SlaError.  Work runs on the first
// tensor's device and its current stream; outputs and scratch memory come from torch's allocator, so a
// captured graph's belong to the graph's own pool.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <sstream>
#include <stdexcept>
#include <string>

#include "sla.h"

namespace {

PyObject *g_error_type = nullptr, *g_memory_type = nullptr;   // SlaError, torch.OutOfMemoryError

struct BadArgument : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Failed {
    sla_status status;
    const char *where;
};

template <class... T>
[[noreturn]] void refuse(const T &...parts)
{
    std::ostringstream s;
    (s << ... << parts);
    throw BadArgument(s.str());
}

std::string shown(const at::Tensor &t)
{
    std::ostringstream s;
    s << t.sizes() << " " << t.scalar_type() << " on " << t.device();
    return s.str();
}

const at::Tensor *tensor(PyObject *o, const char *name)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        refuse(name, ": libsla takes CUDA tensors");
    return &THPVariable_Unpack(o);
}
const at::Tensor &need(PyObject *o, const char *name)
{
    const at::Tensor *t = tensor(o, name);
    if (!t)
        refuse(name, " is needed: libsla takes CUDA tensors");
    return *t;
}

int64_t whole(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(name, " must be a whole number");
    }
    return v;
}

int32_t row_code(const at::Tensor &t)
{
    switch (t.scalar_type()) {
    case at::kFloat: return SLA_F32;
    case at::kDouble: return SLA_F64;
    case at::kBFloat16: return SLA_BF16;
    case at::kHalf: return SLA_F16;
    default: refuse("rows must be float32, float64, bfloat16 or float16, got ", t.scalar_type());
    }
}
// type of states, weights and their gradients
at::ScalarType wide(const at::Tensor &t) { return t.scalar_type() == at::kDouble ? at::kDouble : at::kFloat; }

int32_t gate_code(PyObject *o)
{
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (s && !std::strcmp(s, "value"))
        return SLA_GATE_VALUE;
    if (s && !std::strcmp(s, "exp"))
        return SLA_GATE_EXP;
    if (s && !std::strcmp(s, "sigmoid"))
        return SLA_GATE_SIGMOID;
    refuse("gate must be one of 'exp', 'sigmoid', 'value'", s ? ", got " : "", s ? s : "");
}

// The one stride that walks t's rows ([rows, channels] or [batch, rows, channels]); -1 if there is none.
int64_t row_stride(const at::Tensor &t)
{
    const int64_t dim = t.dim(), d = t.size(dim - 1);
    if (t.numel() == 0)
        return d;
    if (d > 1 && t.stride(dim - 1) != 1)
        return -1;
    int64_t ld, n;
    if (dim == 3) {
        if (t.size(0) == 1) {
            ld = t.stride(1);
            n = t.size(1);
        } else if (t.size(1) == 1) {
            ld = t.stride(0);
            n = t.size(0);
        } else {
            ld = t.stride(1);
            n = 2;
            if (t.stride(0) != t.size(1) * ld)
                return -1;
        }
    } else {
        ld = t.stride(0);
        n = t.size(0);
    }
    if (n <= 1)
        return d;
    return ld >= d || ld == 0 ? ld : -1;
}

// Checks rows against `like` (shape, type, device); their row stride.
int64_t rows(const at::Tensor &t, const at::Tensor &like, const char *name, bool out = false)
{
    if (&t != &like && (t.sizes() != like.sizes() || t.scalar_type() != like.scalar_type() || t.device() != like.device()))
        refuse(name, " must be ", shown(like), ", got ", shown(t));
    const int64_t ld = row_stride(t);
    if (ld < 0)
        refuse(name, ": channels must be contiguous and rows one stride apart");
    if (out && ld < t.size(t.dim() - 1))
        refuse(name, ": an output's rows must not overlap");
    return ld;
}

// The bytes of checked rows: n of `width` bytes, `pitch` apart.
struct Extent {
    uintptr_t first;
    int64_t n, width, pitch;
    explicit Extent(const at::Tensor &t) : first((uintptr_t)t.data_ptr())
    {
        const int64_t d = t.dim() > 0 ? t.size(t.dim() - 1) : 1, ld = t.dim() > 1 ? row_stride(t) : d;
        n = d > 0 ? t.numel() / d : 0;
        if (ld == 0)                                       // one row for all
            n = std::min<int64_t>(n, 1);
        width = d * t.element_size();
        pitch = ld * t.element_size();
    }
    uintptr_t last() const { return first + (uintptr_t)((n - 1) * pitch + width); }
};
bool overlap(const Extent &x, const Extent &y)
{
    if (x.n == 0 || y.n == 0 || x.last() <= y.first || y.last() <= x.first)
        return false;
    if (x.n == 1 ? y.n == 1 : y.n > 1 && x.pitch != y.pitch)
        return true;                                       // two runs of bytes, or rows not told apart
    // columns of one buffer: y's rows start behind x's within the pitch and end before the next one
    const int64_t pitch = x.n > 1 ? x.pitch : y.pitch, apart = (int64_t)(y.first - x.first) % pitch;
    const int64_t at = apart < 0 ? apart + pitch : apart;
    return at < x.width || at + y.width > pitch;
}

// An output may share a buffer with the inputs (columns or other rows of it), but not memory.
void apart(const at::Tensor *out, std::initializer_list<const at::Tensor *> others, const char *name)
{
    for (const at::Tensor *t : others)
        if (out && t && overlap(Extent(*out), Extent(*t)))
            refuse(name, " must not share memory with the other arguments");
}

// Checks a contiguous tensor of the given sizes; its pointer (NULL for none).
void *plain(const at::Tensor *t, at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like, const char *name)
{
    if (!t)
        return nullptr;
    if (t->sizes() != sizes || t->scalar_type() != type || t->device() != like.device())
        refuse(name, " must be ", sizes, " ", type, " on ", like.device(), ", got ", shown(*t));
    if (!t->is_contiguous())
        refuse(name, " must be contiguous");
    return t->data_ptr();
}

// Device and stream of the call, made current while it lives.
struct Place {
    c10::cuda::OptionalCUDAGuard guard;
    at::TensorOptions options;
    void *stream;
    explicit Place(const at::Tensor &t) : options(t.options())
    {
        if (!t.is_cuda())
            refuse("libsla takes CUDA tensors");
        guard.set_device(t.device());
        stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
    }
    at::Tensor make(at::IntArrayRef sizes) const { return at::empty(sizes, options); }
    at::Tensor make(at::IntArrayRef sizes, at::ScalarType type) const { return at::empty(sizes, options.dtype(type)); }
};

// The caller's own tensor was written: autograd's version check has to see that.
void written(const at::Tensor *t)
{
    if (t && !t->is_inference())
        t->unsafeGetTensorImpl()->bump_version();
}

void check(sla_status s, const char *where)
{
    if (s < 0)
        throw Failed{s, where};
}

struct Sequences {
    int64_t tokens, channels;
    int32_t count;
    const int32_t *off;
};
Sequences sequences(const at::Tensor &b, const at::Tensor *seq_off)
{
    if (b.dim() == 3) {
        if (seq_off)
            refuse("seq_off goes with packed [tokens, channels] rows");
        if (b.size(0) > INT32_MAX)
            refuse("too many sequences");
        return {b.size(0) * b.size(1), b.size(2), (int32_t)b.size(0), nullptr};
    }
    if (b.dim() != 2)
        refuse("rows must be [tokens, channels] or [batch, tokens, channels]");
    if (!seq_off)
        return {b.size(0), b.size(1), 1, nullptr};
    if (seq_off->scalar_type() != at::kInt || seq_off->dim() != 1 || seq_off->numel() < 1 || seq_off->device() != b.device() ||
        !seq_off->is_contiguous())
        refuse("seq_off must be a contiguous int32 vector on the rows' device");
    return {b.size(0), b.size(1), (int32_t)(seq_off->numel() - 1), seq_off->data_ptr<int32_t>()};
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
PyObject *wrap_or_none(const at::Tensor &t)
{
    if (t.defined())
        return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
PyObject *tuple(std::initializer_list<PyObject *> items)
{
    PyObject *r = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items)
        PyTuple_SET_ITEM(r, i++, o);
    return r;
}

// ------------------------------------------------------------------ recurrence

// a, b, h0, seq_off, gate, out, h_last -> (h, last)
PyObject *recur_solve(PyObject *const *p)
{
    const at::Tensor &a = need(p[0], "a"), &b = need(p[1], "b");
    const at::Tensor *h0 = tensor(p[2], "h0"), *off = tensor(p[3], "seq_off"), *out = tensor(p[5], "out"),
                     *h_last = tensor(p[6], "h_last");
    const int32_t code = row_code(b), gate = gate_code(p[4]);
    const Sequences q = sequences(b, off);
    const int64_t lda = rows(a, b, "a"), ldb = rows(b, b, "b");
    const int64_t states[2] = {q.count, q.channels};
    void *p0 = plain(h0, states, wide(b), b, "h0");
    int64_t ldh = out ? rows(*out, b, "out", true) : q.channels;
    plain(h_last, states, wide(b), b, "h_last");
    apart(out, {&a, &b, h0, h_last}, "out");
    apart(h_last, {&a, &b, h0}, "h_last");
    const Place here(b);
    const at::Tensor h = out ? *out : here.make(b.sizes());
    const at::Tensor last = h_last ? *h_last : here.make(states, wide(b));
    const size_t size = sla_recur_workspace_bytes(code, q.tokens, q.channels);
    at::Tensor work;
    if (size)
        work = here.make({(int64_t)size}, at::kByte);
    check(sla_recur_solve(code, gate, q.tokens, q.channels, q.count, q.off, a.data_ptr(), lda, b.data_ptr(), ldb, p0,
                          h.data_ptr(), ldh, last.data_ptr(), out ? 0 : SLA_FILL_REST, size ? work.data_ptr() : nullptr,
                          size, here.stream),
          "sla_recur_solve");
    written(out);
    written(h_last);
    return tuple({wrap(h), wrap(last)});
}

// a, h, dh, b, h0, seq_off, dh_last, gate, want_da, want_db, da, db -> (da, db, dh0)
PyObject *recur_adjoint(PyObject *const *p)
{
    const at::Tensor &a = need(p[0], "a"), &h = need(p[1], "h");
    const at::Tensor *dh = tensor(p[2], "dh"), *b = tensor(p[3], "b"), *h0 = tensor(p[4], "h0"), *off = tensor(p[5], "seq_off"),
                     *dlast = tensor(p[6], "dh_last"), *da = tensor(p[10], "da"), *db = tensor(p[11], "db");
    const int32_t code = row_code(h), gate = gate_code(p[7]);
    const bool want_da = PyObject_IsTrue(p[8]) == 1, want_db = PyObject_IsTrue(p[9]) == 1;
    const Sequences q = sequences(h, off);
    const int64_t lda = rows(a, h, "a"), ldh = rows(h, h, "h");
    const bool reads_b = gate == SLA_GATE_SIGMOID && want_da;
    if (reads_b && !b)
        refuse("the sigmoid gate's gradient needs b");
    const int64_t ldb = reads_b ? rows(*b, h, "b") : 0, lddh = dh ? rows(*dh, h, "dh") : 0;
    const int64_t states[2] = {q.count, q.channels};
    void *p0 = plain(h0, states, wide(h), h, "h0"), *plast = plain(dlast, states, wide(h), h, "dh_last");
    const bool given = da || db;
    if (given && ((want_da && !da) || (want_db && !db)))
        refuse("give both da and db, or neither");
    int64_t ldda = want_da && given ? rows(*da, h, "da", true) : q.channels;
    int64_t lddb = want_db && given ? rows(*db, h, "db", true) : q.channels;
    const at::Tensor *to_a = want_da ? da : nullptr, *to_b = want_db ? db : nullptr, *in_b = reads_b ? b : nullptr;
    apart(to_a, {&a, &h, dh, in_b, h0, dlast, to_b}, "da");
    apart(to_b, {&a, &h, dh, in_b, h0, dlast}, "db");
    const Place here(h);
    at::Tensor oa, ob, o0, work;
    if (want_da)
        oa = given ? *da : here.make(h.sizes());
    if (want_db)
        ob = given ? *db : here.make(h.sizes());
    if (h0)
        o0 = here.make(states, wide(h));
    const size_t size = sla_recur_workspace_bytes(code, q.tokens, q.channels);
    if (size)
        work = here.make({(int64_t)size}, at::kByte);
    check(sla_recur_adjoint(code, gate, q.tokens, q.channels, q.count, q.off, a.data_ptr(), lda,
                            reads_b ? b->data_ptr() : nullptr, ldb, h.data_ptr(), ldh, p0, dh ? dh->data_ptr() : nullptr, lddh,
                            plast, want_da ? oa.data_ptr() : nullptr, ldda, want_db ? ob.data_ptr() : nullptr, lddb,
                            h0 ? o0.data_ptr() : nullptr, given ? 0 : SLA_FILL_REST, size ? work.data_ptr() : nullptr, size,
                            here.stream),
          "sla_recur_adjoint");
    written(to_a);
    written(to_b);
    return tuple({wrap_or_none(oa), wrap_or_none(ob), wrap_or_none(o0)});
}

// a, b, state, index, gate, out -> h
PyObject *recur_step(PyObject *const *p)
{
    const at::Tensor &a = need(p[0], "a"), &b = need(p[1], "b"), &state = need(p[2], "state");
    const at::Tensor *index = tensor(p[3], "index"), *out = tensor(p[5], "out");
    const int32_t code = row_code(b), gate = gate_code(p[4]);
    if (b.dim() != 2)
        refuse("rows must be [rows, channels]");
    const int64_t n = b.size(0), channels = b.size(1);
    const int64_t lda = rows(a, b, "a"), ldb = rows(b, b, "b");
    if (state.dim() != 2 || state.size(1) != channels || state.scalar_type() != wide(b) || state.device() != b.device())
        refuse("state must be [slots, ", channels, "] ", wide(b), " on ", b.device(), ", got ", shown(state));
    const int64_t lds = rows(state, state, "state", true);
    if (!index && state.size(0) < n)
        refuse("without index every row needs a slot");
    void *pi = plain(index, {n}, at::kInt, b, "index");
    const int64_t ldh = out ? rows(*out, b, "out", true) : channels;
    apart(out, {&a, &b, &state}, "out");
    apart(&state, {&a, &b}, "state");
    const Place here(b);
    const at::Tensor h = out ? *out : here.make(b.sizes());
    check(sla_recur_step(code, gate, n, channels, state.size(0), a.data_ptr(), lda, b.data_ptr(), ldb, state.data_ptr(), lds,
                         (const int32_t *)pi, h.data_ptr(), ldh, out ? 0 : SLA_FILL_REST, here.stream),
          "sla_recur_step");
    written(&state);
    written(out);
    return wrap(h);
}

// ------------------------------------------------------------------ routing

// expert, n_experts, align, n_slots or None -> (offsets, counts, entry, slot)
PyObject *route_sort(PyObject *const *p)
{
    const at::Tensor &ids = need(p[0], "expert");
    if ((ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong) || (ids.dim() != 1 && ids.dim() != 2) ||
        !ids.is_contiguous())
        refuse("expert must be a contiguous [tokens, top_k] or [tokens] tensor of int32 or int64");
    const int64_t tokens = ids.size(0), top_k = ids.dim() == 1 ? 1 : ids.size(1);
    const int64_t experts = whole(p[1], "n_experts"), align = whole(p[2], "align");
    if (experts < 1 || align < 1 || top_k < 1 || experts > INT32_MAX || align > INT32_MAX || top_k > INT32_MAX)
        refuse("n_experts, align and top_k must be at least 1, and below 2^31");
    const int64_t slots = p[3] == Py_None ? tokens * top_k + experts * (align - 1) : whole(p[3], "n_slots");
    if (slots < 0 || slots > INT32_MAX)
        refuse("n_slots must be within [0, 2^31)");
    const Place here(ids);
    // one allocation, every array on a 16-byte boundary
    const auto up = [](int64_t n) { return (n + 3) / 4 * 4; };
    const int64_t o1 = up(experts + 1), o2 = o1 + up(experts), o3 = o2 + up(slots);
    const at::Tensor buf = here.make({o3 + tokens * top_k}, at::kInt);
    int32_t *base = buf.data_ptr<int32_t>();
    const size_t size = sla_route_workspace_bytes(tokens, (int32_t)top_k, (int32_t)experts);
    at::Tensor work;
    if (size)
        work = here.make({(int64_t)size}, at::kByte);
    check(sla_route_sort(tokens, (int32_t)top_k, (int32_t)experts, (int32_t)align, ids.data_ptr(), (int32_t)ids.element_size(),
                         slots, base, base + o1, base + o2, base + o3, size ? work.data_ptr() : nullptr, size, here.stream),
          "sla_route_sort");
    return tuple({wrap(buf.as_strided({experts + 1}, {1}, 0)), wrap(buf.as_strided({experts}, {1}, o1)),
                  wrap(buf.as_strided({slots}, {1}, o2)), wrap(buf.as_strided({tokens, top_k}, {top_k, 1}, o3))});
}

struct Plan {
    int64_t tokens, slots;
    int32_t top_k, experts;
    const int32_t *offsets, *counts, *slot;
};
Plan route(PyObject *offsets_, PyObject *counts_, PyObject *entry_, PyObject *slot_, const at::Tensor &like)
{
    const at::Tensor &offsets = need(offsets_, "route.offsets"), &counts = need(counts_, "route.counts"),
                     &entry = need(entry_, "route.entry"), &slot = need(slot_, "route.slot");
    if (slot.dim() != 2 || counts.dim() != 1 || entry.dim() != 1)
        refuse("route: slot must be [tokens, top_k], counts and entry vectors");
    const int64_t e = counts.size(0);
    const int32_t *ps = (const int32_t *)plain(&slot, slot.sizes(), at::kInt, like, "route.slot");
    const int32_t *po = (const int32_t *)plain(&offsets, {e + 1}, at::kInt, like, "route.offsets");
    const int32_t *pc = (const int32_t *)plain(&counts, {e}, at::kInt, like, "route.counts");
    return {slot.size(0), entry.size(0), (int32_t)slot.size(1), (int32_t)e, po, pc, ps};
}

// [n, channels] rows of `like`'s type (its own channels where it is the same tensor)
int64_t side(const at::Tensor &t, int64_t n, const at::Tensor &like, const char *name, bool out = false)
{
    if (t.dim() != 2 || t.size(0) != n || like.dim() != 2 || t.size(1) != like.size(1) || t.scalar_type() != like.scalar_type() ||
        t.device() != like.device())
        refuse(name, " must be [", n, ", channels] rows like ", shown(like), ", got ", shown(t));
    return rows(t, t, name, out);
}

// x, offsets, counts, entry, slot, weight, ys, out -> (xs, dweight or None)
PyObject *route_to_slots(PyObject *const *p)
{
    const at::Tensor &x = need(p[0], "rows");
    const int32_t code = row_code(x);
    const Plan r = route(p[1], p[2], p[3], p[4], x);
    const at::Tensor *weight = tensor(p[5], "weight"), *ys = tensor(p[6], "ys"), *out = tensor(p[7], "out");
    const int64_t ldx = side(x, r.tokens, x, "rows"), channels = x.size(1), pairs[2] = {r.tokens, r.top_k};
    void *pw = plain(weight, pairs, wide(x), x, "weight");
    const int64_t ldys = ys ? side(*ys, r.slots, x, "ys") : 0, ldo = out ? side(*out, r.slots, x, "out", true) : channels;
    apart(out, {&x, ys, weight}, "out");
    const Place here(x);
    const at::Tensor xs = out ? *out : here.make({r.slots, channels});
    const uint32_t flags = out ? 0 : SLA_FILL_REST;
    at::Tensor dw;
    if (!ys)
        check(sla_route_dispatch(code, r.tokens, r.top_k, r.experts, r.slots, channels, x.data_ptr(), ldx, r.offsets, r.counts,
                                 r.slot, pw, xs.data_ptr(), ldo, flags, here.stream),
              "sla_route_dispatch");
    else {
        dw = here.make(pairs, wide(x));
        check(sla_route_combine_adjoint(code, r.tokens, r.top_k, r.experts, r.slots, channels, x.data_ptr(), ldx, r.offsets,
                                        r.counts, r.slot, pw, ys->data_ptr(), ldys, xs.data_ptr(), ldo, dw.data_ptr(), flags,
                                        here.stream),
              "sla_route_combine_adjoint");
    }
    written(out);
    return tuple({wrap(xs), wrap_or_none(dw)});
}

// ys, offsets, counts, entry, slot, weight, x, out -> (y, dweight or None)
PyObject *route_to_tokens(PyObject *const *p)
{
    const at::Tensor &ys = need(p[0], "rows");
    const int32_t code = row_code(ys);
    const Plan r = route(p[1], p[2], p[3], p[4], ys);
    const at::Tensor *weight = tensor(p[5], "weight"), *x = tensor(p[6], "x"), *out = tensor(p[7], "out");
    const int64_t ldys = side(ys, r.slots, ys, "rows"), channels = ys.size(1), pairs[2] = {r.tokens, r.top_k};
    void *pw = plain(weight, pairs, wide(ys), ys, "weight");
    const int64_t ldx = x ? side(*x, r.tokens, ys, "x") : 0, ldo = out ? side(*out, r.tokens, ys, "out", true) : channels;
    apart(out, {&ys, x, weight}, "out");
    const Place here(ys);
    const at::Tensor y = out ? *out : here.make({r.tokens, channels});
    at::Tensor dw;
    if (!x)
        check(sla_route_combine(code, r.tokens, r.top_k, r.slots, channels, ys.data_ptr(), ldys, r.slot, pw, y.data_ptr(), ldo,
                                here.stream),
              "sla_route_combine");
    else {
        dw = here.make(pairs, wide(ys));
        check(sla_route_dispatch_adjoint(code, r.tokens, r.top_k, r.slots, channels, ys.data_ptr(), ldys, r.slot, pw,
                                         x->data_ptr(), ldx, y.data_ptr(), ldo, dw.data_ptr(), here.stream),
              "sla_route_dispatch_adjoint");
    }
    written(out);
    return tuple({wrap(y), wrap_or_none(dw)});
}

// t -> its row stride, or None
PyObject *stride_of(PyObject *const *p)
{
    const at::Tensor &t = need(p[0], "rows");
    if (t.dim() != 2 && t.dim() != 3)
        refuse("rows must be [tokens, channels] or [batch, tokens, channels]");
    const int64_t ld = row_stride(t);
    if (ld < 0)
        Py_RETURN_NONE;
    return PyLong_FromLongLong(ld);
}

// x, y -> whether their rows share memory
PyObject *share_memory(PyObject *const *p)
{
    const at::Tensor &x = need(p[0], "x"), &y = need(p[1], "y");
    rows(x, x, "x");
    rows(y, y, "y");
    return PyBool_FromLong(overlap(Extent(x), Extent(y)));
}

PyObject *set_error_types(PyObject *const *p)
{
    Py_INCREF(p[0]);
    Py_XSETREF(g_error_type, p[0]);
    Py_INCREF(p[1]);
    Py_XSETREF(g_memory_type, p[1]);
    Py_RETURN_NONE;
}

// Calls f with its N arguments; no C++ exception leaves it.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        if (n != N)
            refuse("takes ", N, " arguments, got ", n);
        return F(args);
    } catch (const BadArgument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const Failed &e) {
        PyObject *x = PyObject_CallFunction(g_error_type ? g_error_type : PyExc_RuntimeError, "is", (int)e.status, e.where);
        if (x) {
            PyErr_SetObject((PyObject *)Py_TYPE(x), x);
            Py_DECREF(x);
        }
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(g_memory_type ? g_memory_type : PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define ENTRY(f, n) {#f, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(recur_solve, 7), ENTRY(recur_adjoint, 12), ENTRY(recur_step, 6), ENTRY(route_sort, 4),
                           ENTRY(route_to_slots, 8), ENTRY(route_to_tokens, 8), ENTRY(stride_of, 1), ENTRY(share_memory, 2),
                           ENTRY(set_error_types, 2),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_sla_seq", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sla_seq() { return PyModule_Create(&g_module); }
