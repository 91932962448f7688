// Python module `kv_host`: kv.py's and beam.py's calls, from tensors to the C ABI's w12_kv_*
// and w12_beam_select.
//
// A single token's store or attention runs 2 to 7 us on the GPU, and a step makes
// two such calls per layer, so the way to the launch counts.  Looking at the tensors
// (type, shape, strides, device) from Python took 8 us of a 12 us store; here it
// takes well under one.  The checks are made in every call: nothing is remembered
// of a tensor.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <vector>

#include "w12.h"

namespace {

// The C ABI, from the handle that w12.py has on libw12.so, and what raises a status as
// a W12Error.
struct Abi {
    decltype(&w12_kv_plan) plan;
    decltype(&w12_kv_store) store;
    decltype(&w12_kv_read) read;
    decltype(&w12_kv_attend_workspace_size) workspace_size;
    decltype(&w12_kv_attend) attend;
    decltype(&w12_kv_fork_workspace_size) fork_size;
    decltype(&w12_kv_fork) fork;
    decltype(&w12_kv_copy) copy;
    decltype(&w12_kv_attend_shared_workspace_size) shared_size;
    decltype(&w12_kv_attend_shared) attend_shared;
    decltype(&w12_beam_workspace_size) beam_size;
    decltype(&w12_beam_select) beam_select;
    PyObject *raise;
} abi = {};

struct Names {
    PyObject *tables, *lens, *cu_new, *positions, *slots, *max_new, *tree, *owned, *ring, *ring_state, *page_size;
    PyObject *shares, *src, *dst, *rows, *prefix, *cu, *max_requests, *address;
} names;

// An owned reference.
class Ref {
public:
    explicit Ref(PyObject *o) : o_(o) {
        if (!o) throw python_error();
    }
    ~Ref() { Py_DECREF(o_); }
    Ref(const Ref &) = delete;
    Ref &operator=(const Ref &) = delete;
    PyObject *get() const { return o_; }
    PyObject *release() {
        PyObject *o = o_;
        o_ = Py_NewRef(Py_None);
        return o;
    }

private:
    PyObject *o_;
};

Ref field(PyObject *o, PyObject *name) { return Ref(PyObject_GetAttr(o, name)); }

const at::Tensor &tensor(PyObject *o, const char *name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
int32_t int32(int64_t v, const char *name) {
    TORCH_CHECK_VALUE(v >= std::numeric_limits<int32_t>::min() && v <= std::numeric_limits<int32_t>::max(), name,
                      " does not fit 32 bits");
    return static_cast<int32_t>(v);
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return static_cast<float>(v);
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
template <class T>
T *pointer(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw python_error();
    return static_cast<T *>(p);
}

// The elements of a contiguous 1-D tensor on CUDA device `index`.
template <class T>
T *ints(const at::Tensor &t, const char *name, int64_t index) {
    constexpr at::ScalarType type = sizeof(T) == 8 ? at::kLong : at::kInt;
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.dim() == 1 && t.get_device() == index && t.is_contiguous(), name,
                      " must be a contiguous 1-D ", type, " tensor on CUDA device ", index);
    return static_cast<T *>(t.data_ptr());
}

// [tokens, heads * dim] or [tokens, heads, dim] BF16 rows whose heads lie one after
// the other.
struct Rows {
    uint16_t *p = nullptr;
    int64_t stride = 0, tokens = 0, heads = 0;
};
Rows rows(const at::Tensor &t, int64_t dim, const char *name, int64_t index, int64_t heads) {
    Rows r;
    if (t.dim() == 2) {
        if (t.stride(1) == 1 && t.size(1) % dim == 0) r.heads = t.size(1) / dim;
    } else if (t.dim() == 3 && t.size(2) == dim && t.stride(2) == 1 && (t.stride(1) == dim || t.size(1) == 1)) {
        r.heads = t.size(1);
    }
    TORCH_CHECK_VALUE(r.heads >= 1 && t.scalar_type() == at::kBFloat16 && t.get_device() == index &&
                          (heads == 0 || r.heads == heads),
                      name, " must be BF16 [tokens, heads * ", dim, "] on CUDA device ", index,
                      " with contiguous heads", heads ? ", as many as expected" : "");
    r.p = static_cast<uint16_t *>(t.data_ptr());
    r.tokens = t.size(0);
    r.stride = r.tokens > 1 ? t.stride(0) : r.heads * dim;  // one row has no stride that matters
    return r;
}

// Outputs are no part of an autograd graph: they are made, and seen as [tokens, heads,
// dim], without the dispatcher (1000 tokens of an 8-bit cache read into new tensors:
// 4.7 us of host time, 5.9 with at::empty; one token stored into a given `out`: 3.4,
// 6.2 with at::Tensor::view).
at::Tensor new_bf16(at::IntArrayRef sizes, int64_t index) {
    return at::Tensor(at::detail::empty_cuda(sizes, at::kBFloat16,
                                             at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)), {}));
}

at::Tensor by_heads(const at::Tensor &t, const Rows &r, int64_t dim) {
    if (t.dim() == 3) return t;
    at::Tensor view = at::detail::make_tensor<at::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(t.storage()),
                                                              t.key_set(), t.dtype());
    const int64_t sizes[3] = {r.tokens, r.heads, dim}, strides[3] = {t.stride(0), dim, 1};
    view.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(sizes), at::IntArrayRef(strides),
                                                      t.storage_offset());
    return view;
}

void check(int status) {
    if (status == W12_OK) return;
    Ref none(PyObject_CallFunction(abi.raise, "i", status));
    throw std::runtime_error("a W12 call failed");  // unless that raised, as it does
}

template <class F>
void call(F f) {
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f();
    Py_END_ALLOW_THREADS
    check(status);
}

void expect(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "wrong number of arguments"); }

const uint16_t *weight(PyObject *o, int64_t dim, const char *name, int64_t index) {
    if (o == Py_None) return nullptr;
    const at::Tensor &w = tensor(o, name);
    TORCH_CHECK_VALUE(w.scalar_type() == at::kBFloat16 && w.dim() == 1 && w.numel() == dim && w.is_contiguous() &&
                          w.get_device() == index,
                      name, " must be contiguous BF16 [", dim, "] on CUDA device ", index);
    return static_cast<const uint16_t *>(w.data_ptr());
}

// store(cache, index, q, k, v, step, q_norm, k_norm, eps, rope, interleaved, out, stream)
PyObject *store(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 13);
    const w12_kv_cache *c = pointer<const w12_kv_cache>(a[0]);
    const int64_t index = integer(a[1]), dim = c->head_dim;
    const Rows k = rows(tensor(a[3], "k"), dim, "k", index, c->kv_heads);
    const Rows v = rows(tensor(a[4], "v"), dim, "v", index, c->kv_heads);
    const Ref slots_o = field(a[5], names.slots);
    const at::Tensor &slots = tensor(slots_o.get(), "step.slots");
    TORCH_CHECK_VALUE(v.tokens == k.tokens && slots.numel() == k.tokens,
                      "k, v and step.slots must have as many tokens, on the cache's device");
    w12_kv_store_args s = {};
    s.slots = ints<int64_t>(slots, "step.slots", index);
    s.k = k.p, s.k_stride = k.stride;
    s.v = v.p, s.v_stride = v.stride;
    s.tokens = int32(k.tokens, "the number of tokens");
    s.q_norm = weight(a[6], dim, "q_norm", index);
    s.k_norm = weight(a[7], dim, "k_norm", index);
    s.eps = real(a[8]);
    s.interleaved = truth(a[10]);
    if (a[9] != Py_None) {
        const at::Tensor &rope = tensor(a[9], "rope");
        const Ref positions_o = field(a[5], names.positions);
        const at::Tensor &positions = tensor(positions_o.get(), "step.positions");
        TORCH_CHECK_VALUE(rope.scalar_type() == at::kFloat && rope.dim() == 2 && rope.is_contiguous() &&
                              rope.get_device() == index && positions.numel() == k.tokens,
                          "rope must be a contiguous fp32 tensor [positions, rot] on the cache's device and "
                          "step.positions have as many tokens as k");
        s.rope = static_cast<const float *>(rope.data_ptr());
        s.positions = ints<int32_t>(positions, "step.positions", index);
        s.rope_rows = rope.size(0);
        s.rot = int32(rope.size(1), "rope's width");
    }
    void *stream = pointer<void>(a[12]);
    if (a[2] == Py_None) {
        if (s.tokens) call([&] { return abi.store(c, &s, stream); });
        Py_RETURN_NONE;
    }
    const at::Tensor &qt = tensor(a[2], "q");
    const Rows q = rows(qt, dim, "q", index, 0);
    const at::Tensor out = a[11] == Py_None ? new_bf16(qt.sizes(), index) : tensor(a[11], "out");
    const Rows o = rows(out, dim, "out", index, q.heads);
    TORCH_CHECK_VALUE(q.tokens == k.tokens && o.tokens == k.tokens, "q, out and k must have as many tokens");
    s.q = q.p, s.q_stride = q.stride;
    s.q_out = o.p, s.q_out_stride = o.stride;
    s.heads = int32(q.heads, "the number of heads");
    if (s.tokens) call([&] { return abi.store(c, &s, stream); });
    if (out.dim() == 3 && a[11] != Py_None) return Py_NewRef(a[11]);
    return THPVariable_Wrap(by_heads(out, o, dim));
    END_HANDLE_TH_ERRORS
}

// read(cache, index, slots, out, stream)
PyObject *read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 5);
    const w12_kv_cache *c = pointer<const w12_kv_cache>(a[0]);
    const int64_t index = integer(a[1]);
    const at::Tensor &slots = tensor(a[2], "slots");
    const int64_t *at = ints<int64_t>(slots, "slots", index);
    const int32_t tokens = int32(slots.numel(), "the number of tokens");
    const int64_t shape[3] = {tokens, c->kv_heads, c->head_dim};
    at::Tensor to[2];
    PyObject *pair = nullptr;
    if (a[3] == Py_None) {
        to[0] = new_bf16(shape, index);
        to[1] = new_bf16(shape, index);
        Ref k(THPVariable_Wrap(to[0])), v(THPVariable_Wrap(to[1]));
        pair = PyTuple_Pack(2, k.get(), v.get());
    } else {
        pair = PySequence_Tuple(a[3]);
    }
    Ref result(pair);
    TORCH_CHECK_VALUE(PyTuple_GET_SIZE(pair) == 2, "out must be a pair of tensors");
    for (int i = 0; i < 2 && a[3] != Py_None; ++i) {
        to[i] = tensor(PyTuple_GET_ITEM(pair, i), "out");
        TORCH_CHECK_VALUE(to[i].sizes() == at::IntArrayRef(shape) && to[i].scalar_type() == at::kBFloat16 &&
                              to[i].is_contiguous() && to[i].get_device() == index,
                          "out must be two contiguous BF16 tensors [tokens, kv_heads, head_dim]");
    }
    void *stream = pointer<void>(a[4]);
    uint16_t *k = static_cast<uint16_t *>(to[0].data_ptr()), *v = static_cast<uint16_t *>(to[1].data_ptr());
    if (tokens) call([&] { return abi.read(c, at, tokens, k, v, stream); });
    return result.release();
    END_HANDLE_TH_ERRORS
}

// A step's prefix (None: none; so it is for a step that knows of none).
Ref prefix_of(PyObject *step) {
    PyObject *o = PyObject_GetAttr(step, names.prefix);
    if (!o && PyErr_ExceptionMatches(PyExc_AttributeError)) {
        PyErr_Clear();
        o = Py_NewRef(Py_None);
    }
    return Ref(o);
}

// attend(cache, index, q, step, scale, window, out, lse, workspace, grow, stream):
// grow(device, stream, bytes) makes a workspace where `workspace` is None or, found
// by kv.py and not given by the caller (grow not None), too small.
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 11);
    const w12_kv_cache *c = pointer<const w12_kv_cache>(a[0]);
    const int64_t index = integer(a[1]), dim = c->head_dim;
    const at::Tensor &qt = tensor(a[2], "q");
    const Rows q = rows(qt, dim, "q", index, 0);
    const Ref tables_o = field(a[3], names.tables), lens_o = field(a[3], names.lens), cu_o = field(a[3], names.cu_new),
              tree_o = field(a[3], names.tree), new_o = field(a[3], names.max_new),
              positions_o = field(a[3], names.positions);
    const at::Tensor &tables = tensor(tables_o.get(), "step.tables"), &lens = tensor(lens_o.get(), "step.lens"),
                     &cu = tensor(cu_o.get(), "step.cu_new");
    const int64_t requests = lens.numel();
    TORCH_CHECK_VALUE(tables.dim() == 2 && tables.scalar_type() == at::kInt && tables.stride(1) == 1 &&
                          tables.get_device() == index && tables.size(0) == requests && cu.numel() == requests + 1,
                      "step.tables, lens and cu_new must agree and be on the cache's device");
    w12_kv_attend_args s = {};
    s.q = q.p, s.q_stride = q.stride;
    s.tables = static_cast<const int32_t *>(tables.data_ptr());
    s.lens = ints<int32_t>(lens, "step.lens", index);
    s.cu_new = ints<int32_t>(cu, "step.cu_new", index);
    s.requests = int32(requests, "the number of requests");
    s.max_blocks = int32(tables.size(1), "the tables' width");
    s.table_stride = requests > 1 ? tables.stride(0) : tables.size(1);
    s.tokens = int32(q.tokens, "the number of tokens");
    s.heads = int32(q.heads, "the number of heads");
    s.max_new = int32(integer(new_o.get()), "step.max_new");
    s.scale = real(a[4]);
    s.window = int32(integer(a[5]), "window");
    if (tree_o.get() != Py_None) {
        const at::Tensor &tree = tensor(tree_o.get(), "step.tree");
        TORCH_CHECK_VALUE(tree.numel() >= q.tokens, "step.tree must have a mask per token");
        s.tree = reinterpret_cast<const uint32_t *>(ints<int32_t>(tree, "step.tree", index));
        if (s.window > 0 && positions_o.get() != Py_None) {
            const at::Tensor &positions = tensor(positions_o.get(), "step.positions");
            TORCH_CHECK_VALUE(positions.numel() >= q.tokens, "step.positions must have an entry per token");
            s.positions = ints<int32_t>(positions, "step.positions", index);
        }
    }
    if (a[7] != Py_None) {
        const at::Tensor &lse = tensor(a[7], "lse");
        TORCH_CHECK_VALUE(lse.scalar_type() == at::kFloat && lse.dim() == 2 && lse.size(0) == q.tokens &&
                              lse.size(1) == q.heads && lse.is_contiguous() && lse.get_device() == index,
                          "lse must be contiguous fp32 [tokens, heads] on the cache's device");
        s.lse = static_cast<float *>(lse.data_ptr());
    }
    const at::Tensor out = a[6] == Py_None ? new_bf16(qt.sizes(), index) : tensor(a[6], "out");
    const Rows o = rows(out, dim, "out", index, q.heads);
    TORCH_CHECK_VALUE(o.tokens == q.tokens, "out and q must have as many tokens");
    s.out = o.p, s.out_stride = o.stride;
    const Ref prefix_o = prefix_of(a[3]);
    const bool shared = prefix_o.get() != Py_None;
    w12_kv_prefix prefix = {};
    if (shared) {
        const Ref pcu_o = field(prefix_o.get(), names.cu), plens_o = field(prefix_o.get(), names.lens),
                  most_o = field(prefix_o.get(), names.max_requests);
        const at::Tensor &pcu = tensor(pcu_o.get(), "step.prefix.cu"), &plens = tensor(plens_o.get(), "step.prefix.lens");
        prefix.cu = ints<int32_t>(pcu, "step.prefix.cu", index);
        prefix.lens = ints<int32_t>(plens, "step.prefix.lens", index);
        TORCH_CHECK_VALUE(plens.numel() == requests && pcu.numel() >= 2,
                          "step.prefix.lens must have an entry per request and cu one more than groups");
        prefix.groups = int32(pcu.numel() - 1, "the number of groups");
        prefix.max_requests = int32(integer(most_o.get()), "step.prefix.max_requests");
    }
    if (s.tokens) {
        PyObject *ws_o = a[8];
        size_t bytes = 0;
        check(shared ? abi.shared_size(c, &s, &prefix, &bytes) : abi.workspace_size(c, &s, &bytes));
        const auto size = [](PyObject *t) { return tensor(t, "workspace").nbytes(); };
        Ref grown(a[9] != Py_None && (ws_o == Py_None || size(ws_o) < bytes)
                      ? PyObject_CallFunction(a[9], "LOn", static_cast<long long>(index), a[10],
                                              static_cast<Py_ssize_t>(bytes))
                      : Py_NewRef(ws_o));
        const at::Tensor &ws = tensor(grown.get(), "workspace");
        TORCH_CHECK_VALUE(ws.get_device() == index && ws.is_contiguous(),
                          "workspace must be contiguous, on the cache's device");
        void *p = ws.data_ptr(), *stream = pointer<void>(a[10]);
        const size_t have = ws.nbytes();
        call([&] {
            return shared ? abi.attend_shared(c, &s, &prefix, p, have, stream) : abi.attend(c, &s, p, have, stream);
        });
    }
    if (a[6] != Py_None) return Py_NewRef(a[6]);
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// plan(pages, index, lens, new_lens, step, trim, owned_out, ring_state_out, stream)
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 9);
    const int64_t index = integer(a[1]);
    const Ref tables_o = field(a[0], names.tables), owned_o = field(a[0], names.owned),
              ring_o = field(a[0], names.ring), state_o = field(a[0], names.ring_state), page_o = field(a[0], names.page_size),
              cu_o = field(a[4], names.cu_new), positions_o = field(a[4], names.positions),
              slots_o = field(a[4], names.slots);
    const at::Tensor &tables = tensor(tables_o.get(), "tables"), &owned = tensor(owned_o.get(), "owned"),
                     &ring = tensor(ring_o.get(), "ring"), &state = tensor(state_o.get(), "ring_state"),
                     &cu = tensor(cu_o.get(), "step.cu_new"), &positions = tensor(positions_o.get(), "step.positions"),
                     &slots = tensor(slots_o.get(), "step.slots"), &lens = tensor(a[2], "lens"),
                     &fresh = tensor(a[3], "new_lens");
    TORCH_CHECK_VALUE(tables.dim() == 2 && tables.scalar_type() == at::kInt && tables.stride(1) == 1 &&
                          tables.get_device() == index,
                      "tables must be an int32 CUDA tensor [requests, max_blocks] with contiguous rows");
    const int64_t requests = tables.size(0), tokens = slots.numel();
    TORCH_CHECK_VALUE(lens.numel() == requests && fresh.numel() == requests && cu.numel() == requests + 1 &&
                          positions.numel() == tokens && owned.numel() == requests && state.numel() == 2,
                      "lens, new_lens and step must be on the tables' device, with an entry per request");
    w12_kv_plan_args s = {};
    s.lens = ints<int32_t>(lens, "lens", index);
    s.new_lens = ints<int32_t>(fresh, "new_lens", index);
    s.owned_in = s.owned_out = ints<int32_t>(owned, "owned", index);
    s.ring_state_in = s.ring_state_out = ints<int64_t>(state, "ring_state", index);
    if (a[6] != Py_None) {
        const at::Tensor &t = tensor(a[6], "owned_out");
        s.owned_out = ints<int32_t>(t, "owned_out", index);
        TORCH_CHECK_VALUE(t.numel() == requests, "owned_out must have an entry per request");
    }
    if (a[7] != Py_None) {
        const at::Tensor &t = tensor(a[7], "ring_state_out");
        s.ring_state_out = ints<int64_t>(t, "ring_state_out", index);
        TORCH_CHECK_VALUE(t.numel() == 2, "ring_state_out must have two entries");
    }
    s.tables = static_cast<int32_t *>(tables.data_ptr());
    s.table_stride = requests > 1 ? tables.stride(0) : tables.size(1);
    s.ring = ints<int32_t>(ring, "ring", index);
    s.cu_new = ints<int32_t>(cu, "step.cu_new", index);
    s.positions = ints<int32_t>(positions, "step.positions", index);
    s.slots = ints<int64_t>(slots, "step.slots", index);
    s.requests = int32(requests, "the number of requests");
    s.max_blocks = int32(tables.size(1), "the tables' width");
    s.page_size = int32(integer(page_o.get()), "page_size");
    s.ring_size = int32(ring.numel(), "the ring's length");
    s.tokens = int32(tokens, "the number of tokens");
    s.trim = truth(a[5]);
    void *stream = pointer<void>(a[8]);
    call([&] { return abi.plan(&s, stream); });
    return Py_NewRef(a[4]);
    END_HANDLE_TH_ERRORS
}

// fork(pages, index, parents, lens, copies, prefix, lens_out, workspace, grow, stream)
PyObject *fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 10);
    const int64_t index = integer(a[1]);
    const Ref tables_o = field(a[0], names.tables), owned_o = field(a[0], names.owned), ring_o = field(a[0], names.ring),
              state_o = field(a[0], names.ring_state), page_o = field(a[0], names.page_size),
              shares_o = field(a[0], names.shares), src_o = field(a[4], names.src), dst_o = field(a[4], names.dst),
              rows_o = field(a[4], names.rows);
    TORCH_CHECK_VALUE(shares_o.get() != Py_None, "fork needs pages with shares (KVPages.create(..., shared=True))");
    const at::Tensor &tables = tensor(tables_o.get(), "tables"), &owned = tensor(owned_o.get(), "owned"),
                     &ring = tensor(ring_o.get(), "ring"), &state = tensor(state_o.get(), "ring_state"),
                     &shares = tensor(shares_o.get(), "shares"), &parents = tensor(a[2], "parents"),
                     &lens = tensor(a[3], "lens"), &src = tensor(src_o.get(), "copies.src"),
                     &dst = tensor(dst_o.get(), "copies.dst"), &rows = tensor(rows_o.get(), "copies.rows");
    TORCH_CHECK_VALUE(tables.dim() == 2 && tables.scalar_type() == at::kInt && tables.stride(1) == 1 &&
                          tables.get_device() == index,
                      "tables must be an int32 CUDA tensor [requests, max_blocks] with contiguous rows");
    const int64_t requests = tables.size(0);
    TORCH_CHECK_VALUE(parents.numel() == requests && lens.numel() == requests && owned.numel() == requests &&
                          src.numel() == requests && dst.numel() == requests && rows.numel() == requests &&
                          state.numel() == 2,
                      "parents, lens and copies must be on the tables' device, with an entry per request");
    w12_kv_fork_args s = {};
    s.parents = ints<int32_t>(parents, "parents", index);
    s.lens = ints<int32_t>(lens, "lens", index);
    s.owned = ints<int32_t>(owned, "owned", index);
    s.tables = static_cast<int32_t *>(tables.data_ptr());
    s.table_stride = requests > 1 ? tables.stride(0) : tables.size(1);
    s.ring = ints<int32_t>(ring, "ring", index);
    s.ring_state = ints<int64_t>(state, "ring_state", index);
    s.shares = ints<int32_t>(shares, "shares", index);
    s.src = ints<int32_t>(src, "copies.src", index);
    s.dst = ints<int32_t>(dst, "copies.dst", index);
    s.rows = ints<int32_t>(rows, "copies.rows", index);
    s.num_pages = shares.numel();
    s.requests = int32(requests, "the number of requests");
    s.max_blocks = int32(tables.size(1), "the tables' width");
    s.page_size = int32(integer(page_o.get()), "page_size");
    s.ring_size = int32(ring.numel(), "the ring's length");
    if (a[5] != Py_None) {
        const Ref cu_o = field(a[5], names.cu), lens_o = field(a[5], names.lens);
        const at::Tensor &cu = tensor(cu_o.get(), "prefix.cu"), &plens = tensor(lens_o.get(), "prefix.lens");
        s.prefix_cu = ints<int32_t>(cu, "prefix.cu", index);
        s.prefix_lens = ints<int32_t>(plens, "prefix.lens", index);
        TORCH_CHECK_VALUE(plens.numel() == requests && cu.numel() >= 2,
                          "prefix.lens must have an entry per request and cu one more than groups");
        s.groups = int32(cu.numel() - 1, "the number of groups");
    }
    if (a[6] != Py_None) {
        const at::Tensor &t = tensor(a[6], "lens_out");
        s.lens_out = ints<int32_t>(t, "lens_out", index);
        TORCH_CHECK_VALUE(t.numel() == requests, "lens_out must have an entry per request");
    }
    size_t bytes = 0;
    check(abi.fork_size(&s, &bytes));
    Ref grown(a[7] == Py_None || tensor(a[7], "workspace").nbytes() < bytes
                  ? PyObject_CallFunction(a[8], "LOn", static_cast<long long>(index), a[9],
                                          static_cast<Py_ssize_t>(bytes))
                  : Py_NewRef(a[7]));
    const at::Tensor &ws = tensor(grown.get(), "workspace");
    void *p = ws.data_ptr(), *stream = pointer<void>(a[9]);
    const size_t have = ws.nbytes();
    call([&] { return abi.fork(&s, p, have, stream); });
    return Py_NewRef(a[4]);
    END_HANDLE_TH_ERRORS
}

// copy(cache, index, others, copies, stream)
PyObject *copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 5);
    const int64_t index = integer(a[1]);
    std::vector<w12_kv_cache> caches = {*pointer<const w12_kv_cache>(a[0])};
    const Ref others(PySequence_Fast(a[2], "others must be a sequence of caches"));
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(others.get()); ++i) {
        const Ref address = field(PySequence_Fast_GET_ITEM(others.get(), i), names.address);
        caches.push_back(*pointer<const w12_kv_cache>(address.get()));
    }
    const Ref src_o = field(a[3], names.src), dst_o = field(a[3], names.dst), rows_o = field(a[3], names.rows);
    const at::Tensor &src = tensor(src_o.get(), "copies.src"), &dst = tensor(dst_o.get(), "copies.dst");
    const int32_t *from = ints<int32_t>(src, "copies.src", index), *to = ints<int32_t>(dst, "copies.dst", index);
    const int32_t *rows = nullptr;
    TORCH_CHECK_VALUE(src.numel() == dst.numel(), "copies must have as many src as dst");
    if (rows_o.get() != Py_None) {
        const at::Tensor &t = tensor(rows_o.get(), "copies.rows");
        rows = ints<int32_t>(t, "copies.rows", index);
        TORCH_CHECK_VALUE(t.numel() == src.numel(), "copies must have as many rows as src");
    }
    const int32_t pairs = int32(src.numel(), "the number of copies");
    void *stream = pointer<void>(a[4]);
    if (pairs)
        call([&] { return abi.copy(caches.data(), (int32_t)caches.size(), from, to, rows, pairs, stream); });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// select(args, index, logits, allowed, scores, workspace, grow, stream): args is the
// holder's struct with its outputs; logits [requests * beams, vocab] or [requests, beams, vocab]
PyObject *select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 8);
    w12_beam_args s = *pointer<const w12_beam_args>(a[0]);
    const int64_t index = integer(a[1]), rows = (int64_t)s.requests * s.beams;
    const at::Tensor &logits = tensor(a[2], "logits");
    bool good = logits.get_device() == index &&
                (logits.scalar_type() == at::kBFloat16 || logits.scalar_type() == at::kFloat);
    if (good && logits.dim() == 2) {
        good = logits.size(0) == rows;
        s.logits_stride = rows > 1 ? logits.stride(0) : logits.size(1);
    } else {
        good = good && logits.dim() == 3 && logits.size(0) == s.requests && logits.size(1) == s.beams;
        if (good) {
            s.logits_stride = s.beams > 1 ? logits.stride(1) : s.requests > 1 ? logits.stride(0) : logits.size(2);
            good = s.requests == 1 || logits.stride(0) == s.beams * s.logits_stride;
        }
    }
    good = good && (logits.stride(-1) == 1 || logits.size(-1) == 1);
    TORCH_CHECK_VALUE(good, "logits must be BF16 or fp32 [", rows, ", vocab] on CUDA device ", index,
                      " with contiguous rows");
    s.logits = logits.data_ptr();
    s.dtype = logits.scalar_type() == at::kBFloat16 ? W12_BEAM_BF16 : W12_BEAM_F32;
    s.vocab = int32(logits.size(-1), "the vocabulary");
    if (a[3] != Py_None) {
        const at::Tensor &t = tensor(a[3], "allowed");
        const int64_t words = (s.vocab + 31LL) / 32;
        const bool one = t.dim() == 1;
        TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.get_device() == index && (one || t.dim() == 2) &&
                              t.size(-1) == words && (t.stride(-1) == 1 || words == 1) && (one || t.size(0) == rows),
                          "allowed must be int32 [", rows, ", ", words, "] or [", words, "] on CUDA device ", index,
                          " with contiguous rows");
        s.allowed = static_cast<const uint32_t *>(t.data_ptr());
        s.allowed_stride = one ? 0 : rows > 1 ? t.stride(0) : words;
        TORCH_CHECK_VALUE(one || s.allowed_stride >= words, "allowed's rows overlap");
    }
    if (a[4] != Py_None) {
        const at::Tensor &t = tensor(a[4], "scores");
        TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && t.get_device() == index && t.numel() == rows &&
                              t.is_contiguous(),
                          "scores must be contiguous fp32 [requests, beams] on CUDA device ", index);
        s.scores_in = static_cast<const float *>(t.data_ptr());
    }
    size_t bytes = 0;
    check(abi.beam_size(&s, &bytes));
    Ref grown(a[5] == Py_None || tensor(a[5], "workspace").nbytes() < bytes
                  ? PyObject_CallFunction(a[6], "LOn", static_cast<long long>(index), a[7],
                                          static_cast<Py_ssize_t>(bytes))
                  : Py_NewRef(a[5]));
    const at::Tensor &ws = tensor(grown.get(), "workspace");
    void *p = ws.data_ptr(), *stream = pointer<void>(a[7]);
    const size_t have = ws.nbytes();
    call([&] { return abi.beam_select(&s, p, have, stream); });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// bind(plan, store, read, workspace_size, attend, fork_size, fork, copy, shared_size, attend_shared,
// beam_size, beam_select, raise): the C ABI's addresses
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 13);
    const auto set = [](auto &f, PyObject *o) { f = reinterpret_cast<std::decay_t<decltype(f)>>(pointer<void>(o)); };
    set(abi.plan, a[0]);
    set(abi.store, a[1]);
    set(abi.read, a[2]);
    set(abi.workspace_size, a[3]);
    set(abi.attend, a[4]);
    set(abi.fork_size, a[5]);
    set(abi.fork, a[6]);
    set(abi.copy, a[7]);
    set(abi.shared_size, a[8]);
    set(abi.attend_shared, a[9]);
    set(abi.beam_size, a[10]);
    set(abi.beam_select, a[11]);
    Py_XDECREF(abi.raise);
    abi.raise = Py_NewRef(a[12]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define W12_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"plan", W12_FAST(plan)},     {"store", W12_FAST(store)}, {"read", W12_FAST(read)},
                         {"attend", W12_FAST(attend)}, {"fork", W12_FAST(fork)},   {"copy", W12_FAST(copy)},
                         {"select", W12_FAST(select)}, {"bind", W12_FAST(bind)},   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kv_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kv_host() {
    const auto name = [](const char *s) { return PyUnicode_InternFromString(s); };
    names = {name("tables"), name("lens"), name("cu_new"), name("positions"), name("slots"), name("max_new"),
             name("tree"), name("owned"), name("ring"), name("ring_state"), name("page_size"), name("shares"),
             name("src"), name("dst"), name("rows"), name("prefix"), name("cu"), name("max_requests"),
             name("_address")};
    return PyModule_Create(&module);
}
