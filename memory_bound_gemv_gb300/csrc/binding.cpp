// The common case of the decode-step calls' Python binding: checks of the
// tensors, packing of the argument structures and the call, in one step.
//
// A decode step's small calls take 2 to 3 us on the GPU; reading a dozen
// tensors' types, shapes and strides from Python takes 5 us and more.  Every
// function here answers the C status of the call, or -1 where something is
// not as the common case has it: decode.py then goes through its own checks,
// which name what is wrong.  Nothing is decided here alone, and nothing is kept
// between calls.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "../../include/gemv.h"

namespace {

gemv_status_t (*p_attn)(const gemv_kv_t *, const gemv_attn_t *, int, void *);
gemv_status_t (*p_rope)(const gemv_kv_t *, const gemv_rope_t *, void *);
gemv_status_t (*p_rope_norm)(const gemv_kv_t *, const gemv_rope_t *, const gemv_head_norm_t *, void *);
gemv_status_t (*p_assign)(const gemv_kv_t *, const gemv_assign_t *, void *);
gemv_status_t (*p_plan)(const gemv_kv_t *, const int32_t *, int, int, int, int32_t *, int64_t, int32_t *, void *);
gemv_status_t (*p_apply)(const gemv_kv_t *, const int32_t *, int64_t, const int32_t *, int32_t *, int, void *);
gemv_status_t (*p_norm)(const gemv_norm_t *, void *);

// Not the common case.
struct Other {};

int elem_of(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return GEMV_ELEM_F32;
    case at::kHalf: return GEMV_ELEM_F16;
    case at::kBFloat16: return GEMV_ELEM_BF16;
    default: throw Other();
    }
}

at::ScalarType type_of(int elem) { return elem == GEMV_ELEM_F16 ? at::kHalf : at::kBFloat16; }

const at::Tensor &tensor(PyObject *o, int64_t index)
{
    if (!THPVariable_Check(o)) throw Other();
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != index) throw Other();
    return t;
}

// A tensor of this type and shape whose last dimension is contiguous.
const at::Tensor &operand(PyObject *o, int64_t index, at::ScalarType type, std::initializer_list<int64_t> shape)
{
    const at::Tensor &t = tensor(o, index);
    if (t.scalar_type() != type || t.dim() != static_cast<int64_t>(shape.size())) throw Other();
    int64_t d = 0;
    for (int64_t n : shape)
        if (t.size(d++) != n) throw Other();
    if (t.size(d - 1) > 1 && t.stride(d - 1) != 1) throw Other();
    return t;
}

// The address of a contiguous int32 or float32 tensor of this shape.
template <typename T>
T *dense(PyObject *o, int64_t index, std::initializer_list<int64_t> shape)
{
    const at::Tensor &t = operand(o, index, std::is_same<T, float>::value ? at::kFloat : at::kInt, shape);
    if (!t.is_contiguous()) throw Other();
    return static_cast<T *>(t.data_ptr());
}

gemv_heads_t heads(const at::Tensor &t) { return {t.data_ptr(), {t.stride(0), t.stride(1)}}; }

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Other();
    }
    return v;
}

int32_t integer32(PyObject *o)
{
    const int64_t v = integer(o);
    if (v != static_cast<int32_t>(v)) throw Other();
    return static_cast<int32_t>(v);
}

float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Other();
    }
    return static_cast<float>(v);
}

const gemv_kv_t *cache(PyObject *o) { return reinterpret_cast<const gemv_kv_t *>(integer(o)); }

// The stream given as a handle, or the current one.
void *stream_of(PyObject *o, int64_t index)
{
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    return reinterpret_cast<void *>(integer(o));
}

template <typename F>
PyObject *answer(Py_ssize_t n, Py_ssize_t wanted, F call)
{
    int status = -1;
    if (n == wanted) {
        try {
            status = call();
        } catch (const Other &) {
        } catch (const std::exception &) {  // torch's own refusals: the slow path words them
        }
    }
    return PyLong_FromLong(status);
}

// (cache, device, q, lengths, out, lse, scores_out address, workspace address, its bytes, scale, window, stream), and sinks (0)
PyObject *attn(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer(n == 13 ? 12 : n, 12, [&]() -> int {
        const gemv_kv_t *kv = cache(a[0]);
        const int64_t index = integer(a[1]);
        gemv_attn_t g;
        std::memset(&g, 0, sizeof(g));
        const at::Tensor &q = tensor(a[2], index);
        if (q.dim() != 3) throw Other();
        const int64_t count = q.size(1);
        if (count < 1 || kv->kv_heads < 1 || count % kv->kv_heads || count > INT32_MAX) throw Other();
        const at::ScalarType type = type_of(kv->elem);
        g.q = heads(operand(a[2], index, type, {kv->batch, count, kv->head_dim}));
        g.lengths = dense<int32_t>(a[3], index, {kv->batch});
        g.out = heads(operand(a[4], index, type, {kv->batch, count, kv->head_dim}));
        if (a[5] != Py_None) g.lse = dense<float>(a[5], index, {kv->batch, count});
        g.scores_out = reinterpret_cast<float *>(integer(a[6]));
        g.workspace = reinterpret_cast<void *>(integer(a[7]));
        g.workspace_bytes = static_cast<size_t>(integer(a[8]));
        g.q_heads = static_cast<int32_t>(count);
        g.scale = real(a[9]);
        g.window = integer32(a[10]);
        const int sinks = n == 13 ? integer32(a[12]) : 0;
        if (g.window < 0 || sinks < 0) throw Other();
        return p_attn(kv, &g, sinks, stream_of(a[11], index));
    });
}

// A norm's weight [dim] of any type; None: NULL.
const void *weight_of(PyObject *o, int64_t index, int64_t dim, int32_t *elem)
{
    *elem = GEMV_ELEM_F32;
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, index);
    *elem = elem_of(t.scalar_type());
    return operand(o, index, t.scalar_type(), {dim}).data_ptr();
}

// (cache, device, rope's packed fields, q, k, v, positions, slots, seq, stamps, q_out, stream), and for norms
// (q_weight, k_weight, unit_offset, eps) behind them
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer(n == 16 ? 12 : n, 12, [&]() -> int {
        const gemv_kv_t *kv = cache(a[0]);
        const int64_t index = integer(a[1]);
        gemv_rope_t g;
        std::memset(&g, 0, sizeof(g));
        struct {
            uint64_t turns, axis;
            int32_t index, axes, rot, pairs;
        } r;
        if (!PyBytes_Check(a[2]) || PyBytes_GET_SIZE(a[2]) != sizeof(r)) throw Other();
        std::memcpy(&r, PyBytes_AS_STRING(a[2]), sizeof(r));
        const at::Tensor &q = tensor(a[3], index);
        if (q.dim() != 3 || r.index != index || r.rot > kv->head_dim) throw Other();
        const int64_t tokens = q.size(0), count = q.size(1);
        if (tokens > INT32_MAX || count > INT32_MAX) throw Other();
        const at::ScalarType type = q.scalar_type();
        g.src_elem = elem_of(type);
        g.q = heads(operand(a[3], index, type, {tokens, count, kv->head_dim}));
        g.k = heads(operand(a[4], index, type, {tokens, kv->kv_heads, kv->head_dim}));
        g.v = heads(operand(a[5], index, type, {tokens, kv->kv_heads, kv->head_dim}));
        const at::Tensor &pos = operand(a[6], index, at::kInt, {r.axes, tokens});
        g.positions = static_cast<const int32_t *>(pos.data_ptr());
        g.pos_stride = pos.stride(0);
        g.slots = dense<int32_t>(a[7], index, {tokens});
        if (a[8] != Py_None)
            g.seq = dense<int32_t>(a[8], index, {tokens});
        else if (tokens > kv->batch)
            throw Other();
        if (a[9] != Py_None) g.stamps = dense<int32_t>(a[9], index, {tokens});
        g.q_out = heads(operand(a[10], index, type_of(kv->elem), {tokens, count, kv->head_dim}));
        g.turns = reinterpret_cast<const uint64_t *>(r.turns);
        g.axis = reinterpret_cast<const uint8_t *>(r.axis);
        g.tokens = static_cast<int32_t>(tokens);
        g.q_heads = static_cast<int32_t>(count);
        g.axes = r.axes;
        g.rot = r.rot;
        g.pairs = r.pairs;
        if (n == 12) return p_rope(kv, &g, stream_of(a[11], index));
        gemv_head_norm_t w;
        w.q_weight = weight_of(a[12], index, kv->head_dim, &w.q_elem);
        w.k_weight = weight_of(a[13], index, kv->head_dim, &w.k_elem);
        w.unit_offset = integer(a[14]) != 0;
        w.eps = real(a[15]);
        return p_rope_norm(kv, &g, &w, stream_of(a[11], index));
    });
}

// Room of a moves tensor [batch, kv_heads, room, 2].
int64_t room_of(const gemv_kv_t *kv, PyObject *o, int64_t index, int32_t **moves)
{
    const at::Tensor &t = tensor(o, index);
    if (t.dim() != 4) throw Other();
    *moves = dense<int32_t>(o, index, {kv->batch, kv->kv_heads, t.size(2), 2});
    return t.size(2);
}

// (cache, device, lengths, keep, sinks, recent, moves, counts, stream)
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer(n, 9, [&]() -> int {
        const gemv_kv_t *kv = cache(a[0]);
        const int64_t index = integer(a[1]);
        const int32_t *lengths = dense<int32_t>(a[2], index, {kv->batch});
        const int keep = integer32(a[3]), sinks = integer32(a[4]), recent = integer32(a[5]);
        int32_t *moves;
        const int64_t room = room_of(kv, a[6], index, &moves);
        int32_t *counts = dense<int32_t>(a[7], index, {kv->batch, kv->kv_heads});
        const int64_t behind = static_cast<int64_t>(kv->max_pages) * kv->page_size - keep;
        const int64_t most = behind < keep ? behind : keep;
        if (keep < 1 || sinks < 0 || recent < 0 || room < 1 || room < most || !kv->scores || !kv->stamps) throw Other();
        return p_plan(kv, lengths, keep, sinks, recent, moves, room, counts, stream_of(a[8], index));
    });
}

// (cache, device, moves, counts, lengths, keep, stream)
PyObject *apply(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer(n, 7, [&]() -> int {
        const gemv_kv_t *kv = cache(a[0]);
        const int64_t index = integer(a[1]);
        int32_t *moves;
        const int64_t room = room_of(kv, a[2], index, &moves);
        int32_t *counts = dense<int32_t>(a[3], index, {kv->batch, kv->kv_heads});
        int32_t *lengths = a[4] == Py_None ? nullptr : dense<int32_t>(a[4], index, {kv->batch});
        const int keep = integer32(a[5]);
        if (keep < 1) throw Other();
        return p_apply(kv, moves, room, counts, lengths, keep, stream_of(a[6], index));
    });
}

// (cache, device, ring, state, lengths, fresh, starts, slots, seq, shared, lengths_out, state_out, stream)
PyObject *assign(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer(n, 13, [&]() -> int {
        const gemv_kv_t *kv = cache(a[0]);
        const int64_t index = integer(a[1]);
        gemv_assign_t g;
        std::memset(&g, 0, sizeof(g));
        const at::Tensor &ring = tensor(a[2], index), &slots = tensor(a[7], index);
        if (ring.dim() != 1 || slots.dim() != 1) throw Other();
        g.ring_size = ring.size(0);
        g.room = slots.size(0);
        g.ring = dense<int32_t>(a[2], index, {g.ring_size});
        g.state = dense<int32_t>(a[3], index, {2});
        g.lengths = dense<int32_t>(a[4], index, {kv->batch});
        g.fresh = dense<int32_t>(a[5], index, {kv->batch});
        g.starts = dense<int32_t>(a[6], index, {kv->batch + 1});
        g.slots = dense<int32_t>(a[7], index, {g.room});
        g.seq = dense<int32_t>(a[8], index, {g.room});
        if (a[9] != Py_None) g.shared = dense<int32_t>(a[9], index, {kv->batch});
        g.lengths_out = a[10] == Py_None ? const_cast<int32_t *>(g.lengths) : dense<int32_t>(a[10], index, {kv->batch});
        g.state_out = a[11] == Py_None ? const_cast<int32_t *>(g.state) : dense<int32_t>(a[11], index, {2});
        return p_assign(kv, &g, stream_of(a[12], index));
    });
}

gemv_rows_t rows_of(PyObject *o, int64_t index, int64_t rows, int64_t width, bool one_row)
{
    if (o == Py_None) return {nullptr, 0, 0};
    const at::Tensor &t = tensor(o, index);
    const int elem = elem_of(t.scalar_type());
    if (one_row && t.dim() == 1) {
        operand(o, index, t.scalar_type(), {width});
        return {t.data_ptr(), 0, elem};
    }
    operand(o, index, t.scalar_type(), {rows, width});
    return {t.data_ptr(), t.stride(0), elem};
}

// (y, x, gate, post_weight, pre_weight, pre_bias, out, h, alpha, eps, flags, stream)
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer(n, 12, [&]() -> int {
        if (!THPVariable_Check(a[0])) throw Other();
        const at::Tensor &y = THPVariable_Unpack(a[0]);
        if (!y.defined() || !y.is_cuda() || y.dim() != 2) throw Other();
        const int64_t index = y.get_device(), rows = y.size(0), width = y.size(1);
        gemv_norm_t g;
        std::memset(&g, 0, sizeof(g));
        g.y = rows_of(a[0], index, rows, width, false);
        g.x = rows_of(a[1], index, rows, width, false);
        g.gate = rows_of(a[2], index, rows, width, true);
        g.post_weight = rows_of(a[3], index, rows, width, true);
        g.pre_weight = rows_of(a[4], index, rows, width, true);
        g.pre_bias = rows_of(a[5], index, rows, width, true);
        g.out = rows_of(a[6], index, rows, width, false);
        g.h = rows_of(a[7], index, rows, width, false);
        if (!g.x.data || !g.out.data || g.out.elem != g.x.elem) throw Other();
        g.rows = rows;
        g.width = width;
        g.alpha = real(a[8]);
        g.eps = real(a[9]);
        g.flags = static_cast<uint32_t>(integer(a[10]));
        return p_norm(&g, stream_of(a[11], index));
    });
}

// The library's entry points: (attn, rope, plan, apply, norm, rope with norms, assign) as addresses.
PyObject *use(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    long long at[7] = {0, 0, 0, 0, 0, 0, 0};
    for (Py_ssize_t i = 0; i < 7 && i < n; ++i) at[i] = PyLong_AsLongLong(a[i]);
    if (PyErr_Occurred()) return nullptr;
    p_attn = reinterpret_cast<decltype(p_attn)>(at[0]);
    p_rope = reinterpret_cast<decltype(p_rope)>(at[1]);
    p_plan = reinterpret_cast<decltype(p_plan)>(at[2]);
    p_apply = reinterpret_cast<decltype(p_apply)>(at[3]);
    p_norm = reinterpret_cast<decltype(p_norm)>(at[4]);
    p_rope_norm = reinterpret_cast<decltype(p_rope_norm)>(at[5]);
    p_assign = reinterpret_cast<decltype(p_assign)>(at[6]);
    Py_RETURN_NONE;
}

#define MBG_FUNCTION(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef functions[] = {MBG_FUNCTION(attn), MBG_FUNCTION(rope), MBG_FUNCTION(plan), MBG_FUNCTION(apply),
                           MBG_FUNCTION(norm), MBG_FUNCTION(assign), MBG_FUNCTION(use), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mbgbinding", nullptr, -1, functions, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mbgbinding()
{
    PyObject *m = PyModule_Create(&module);
    // what it was compiled for
    if (m) PyModule_AddStringConstant(m, "torch_version", MBG_TORCH_VERSION);
    return m;
}
