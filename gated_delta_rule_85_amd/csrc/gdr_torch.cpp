// Python binding of the operators on a pool of states: the argument checks of
// pool.py's functions and the calls of libgdr.
//
// A decode step calls these once per layer and token, on kernels of 5 us.  A call takes the
// host 4.3 us here, 2.4 of them the launch; with the same checks in Python it took 9.6.  The
// module holds no state but the two Python objects that pool.py hands it; every operation
// runs in libgdr's kernels.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "gdr.h"

namespace {

PyObject *library_error = nullptr;  // GdrError(entry point, code)
PyObject *current_stream = nullptr; // device index -> handle of its current stream

#define NEED(cond, ...) TORCH_CHECK_VALUE(cond, __VA_ARGS__)

const at::Tensor *optional_tensor(PyObject *o, const char *name) {
    if (o == Py_None) return nullptr;
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor &tensor(PyObject *o, const char *name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

int element(at::ScalarType t) { return t == at::kBFloat16 ? GDR_BF16 : t == at::kFloat ? GDR_F32 : -1; }
bool aligned(const at::Tensor &t) { return ((uintptr_t)t.data_ptr() & 15) == 0; }
bool overlap(const at::Tensor &a, const at::Tensor &b) {
    if (a.device() != b.device() || a.numel() == 0 || b.numel() == 0) return false;
    auto span = [](const at::Tensor &t) {
        int64_t last = 0;
        for (int64_t d = 0; d < t.dim(); ++d) last += (t.size(d) - 1) * t.stride(d);
        return (last + 1) * t.element_size();
    };
    const char *x = (const char *)a.data_ptr(), *y = (const char *)b.data_ptr();
    return x < y + span(b) && y < x + span(a);
}

// A tensor as the kernels read it, kept alive by `held` where it had to be made
struct Held {
    at::Tensor made[9];  // at most: q, k, v, g, beta and four index arrays
    int n = 0;
    const at::Tensor &keep(at::Tensor t) { return made[n++] = std::move(t); }
};

// q, k or v with the elements between its tokens and between its batch rows, copied if the
// kernels cannot read it in place: they need one token's [H, D] contiguous and rows at
// multiples of 16 bytes, less than 2^23 elements apart
struct Rows {
    const void *data;
    int64_t row, batch;
};
Rows rows(const at::Tensor &x, Held &held) {
    const int64_t B = x.size(0), T = x.size(1), H = x.size(2), D = x.size(3), per16 = 16 / x.element_size();
    const int64_t batch = B < 2 ? 0 : x.stride(0), row = T < 2 ? 0 : x.stride(1);
    if (x.stride(3) == 1 && (H < 2 || x.stride(2) == D) && batch % per16 == 0 && row % per16 == 0 && row < 1 << 23 &&
        aligned(x))
        return {x.data_ptr(), row, batch};
    return {held.keep(x.clone(at::MemoryFormat::Contiguous)).data_ptr(), H * D, T * H * D};
}
const float *floats(const at::Tensor &x, Held &held) {
    if (x.scalar_type() == at::kFloat && x.is_contiguous()) return x.const_data_ptr<float>();
    return held.keep(x.to(at::kFloat).contiguous()).const_data_ptr<float>();
}
// an index array where the kernels read it
const int32_t *indices(const at::Tensor *x, const at::Device &dev, Held &held) {
    if (!x) return nullptr;
    if (x->device() == dev && x->is_contiguous()) return x->const_data_ptr<int32_t>();
    return held.keep(x->to(x->options().device(dev)).contiguous()).const_data_ptr<int32_t>();
}

// An int32 index array of n entries; on the host its range [lo, hi) is checked
void check_indices(const at::Tensor &x, int64_t n, const char *what, int64_t lo, int64_t hi) {
    NEED(x.scalar_type() == at::kInt && x.dim() == 1 && x.numel() == n, what, " must be int32 [", n, "]");
    if (x.is_cuda()) return;
    const at::Tensor c = x.contiguous();
    const int32_t *p = c.const_data_ptr<int32_t>();
    for (int64_t i = 0; i < n; ++i) NEED(p[i] >= lo && p[i] < hi, what, " out of range [", lo, ", ", hi, ")");
}
void check_distinct(const at::Tensor &slots) {
    const at::Tensor c = slots.contiguous();
    const int32_t *p = c.const_data_ptr<int32_t>();
    std::vector<int32_t> used;
    for (int64_t i = 0; i < c.numel(); ++i)
        if (p[i] >= 0) used.push_back(p[i]);
    std::sort(used.begin(), used.end());
    NEED(std::adjacent_find(used.begin(), used.end()) == used.end(), "slots names a slot twice");
}
void check_offsets(const at::Tensor &cu, int64_t T) {
    const at::Tensor c = cu.contiguous();
    const int32_t *p = c.const_data_ptr<int32_t>();
    const int64_t n = c.numel();
    bool ok = n >= 2 && p[0] == 0 && p[n - 1] == T;
    for (int64_t i = 1; i < n; ++i) ok = ok && p[i] >= p[i - 1];
    NEED(ok, "cu_seqlens must start at 0, never decrease and end at T");
}
// (the offsets, where on the host, have been checked)
void check_parents(const at::Tensor &parents, int64_t B, int64_t T, const at::Tensor *cu) {
    NEED(parents.scalar_type() == at::kInt && parents.dim() == 2 && parents.size(0) == B && parents.size(1) == T,
         "parents must be int32 [B,T]");
    NEED(cu || T <= GDR_TREE_MAX, "a tree has at most ", GDR_TREE_MAX, " nodes");
    if (cu && cu->is_cuda()) return;
    const at::Tensor c = cu ? cu->contiguous() : at::Tensor(), p = parents.is_cuda() ? at::Tensor() : parents.contiguous();
    const int64_t n_seq = cu ? c.numel() - 1 : B;
    for (int64_t j = 0; j < n_seq; ++j) {
        const int64_t b = cu ? c.const_data_ptr<int32_t>()[j] : j * T, e = cu ? c.const_data_ptr<int32_t>()[j + 1] : b + T;
        NEED(e - b <= GDR_TREE_MAX, "a tree has at most ", GDR_TREE_MAX, " nodes");
        if (p.defined())
            for (int64_t i = b; i < e; ++i) {
                const int32_t up = p.const_data_ptr<int32_t>()[i];
                NEED(up >= -1 && up < i - b, "a node's parent is -1 or an earlier node of its tree");
            }
    }
}
void check_accepted(const at::Tensor &accepted, int64_t n_seq, int64_t T, const at::Tensor *cu) {
    check_indices(accepted, n_seq, "accepted", -1, cu ? GDR_TREE_MAX : T);
    if (!cu || cu->is_cuda() || accepted.is_cuda()) return;
    const at::Tensor c = cu->contiguous(), a = accepted.contiguous();
    const int32_t *offsets = c.const_data_ptr<int32_t>(), *nodes = a.const_data_ptr<int32_t>();
    for (int64_t j = 0; j < n_seq; ++j)
        NEED(nodes[j] < offsets[j + 1] - offsets[j], "accepted is -1 or a node of its tree");
}
// Refuses what autograd would have to follow.  (torch.no_grad() leaves forward mode on.)
struct NoGradient {
    const bool backward = at::GradMode::is_enabled(), forward = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    void check(const at::Tensor &t) const {
        if (!t.unsafeGetTensorImpl()->autograd_meta()) return;  // as on most tensors: neither of them
        NEED(!backward || !t.requires_grad(), "the operators on a pool of states have no gradient: use "
                                              "chunk_gated_delta_rule, or torch.no_grad()");
        NEED(!forward || !t._fw_grad(0).defined(),
             "the operators on a pool of states have no gradient, and no tangent in forward mode");
    }
};
// a pool's slots: each contiguous and aligned, apart from each other
void check_slots(const at::Tensor &states, int64_t first, const char *name) {
    const int64_t n = states.size(first), H = states.size(first + 1), K = states.size(first + 2), V = states.size(first + 3);
    NEED(n >= 1 && states.stride(first + 3) == 1 && states.stride(first + 2) == V &&
             (H < 2 || states.stride(first + 1) == K * V) && aligned(states) &&
             (n < 2 || (states.stride(first) % 4 == 0 && states.stride(first) >= H * K * V)),
         "a slot of ", name, " must be contiguous and 16-byte aligned");
}

// Runs an entry point on the device's current stream.  What the kernels write in place is
// `written`: autograd is told, so that a backward that has saved it raises an error instead of
// using the new values.  False: a Python error is set.
template <typename Args>
bool launch(int (*entry)(const Args *, hipStream_t), const char *name, const Args &args, const at::Device &dev,
            std::initializer_list<const at::Tensor *> written) {
    const c10::DeviceGuard guard(dev);
    PyObject *index = PyLong_FromLong(dev.index()), *handle = nullptr;
    if (index) handle = PyObject_CallOneArg(current_stream, index);
    Py_XDECREF(index);
    if (!handle) return false;
    void *stream = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!stream && PyErr_Occurred()) return false;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = entry(&args, (hipStream_t)stream);
    Py_END_ALLOW_THREADS
    if (rc) {
        PyObject *e = PyObject_CallFunction(library_error, "si", name, rc);
        if (e) PyErr_SetObject(library_error, e);
        Py_XDECREF(e);
        return false;
    }
    for (const at::Tensor *t : written)
        if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
    return true;
}

enum class Op { STEP, TREE, ACCEPT };

struct Call {
    const at::Tensor *q, *k, *v, *g, *beta, *parents, *accepted, *states, *cu, *slots, *out;
    PyObject *scale, *output_dtype;
};

// Checks the arguments and launches; `o` receives the output.  False: a Python error is set.
bool run(Op op, const Call &x, at::Tensor &o) {
    const at::Tensor &k = *x.k, &v = *x.v, &states = *x.states;
    NEED(k.dim() == 4 && v.dim() == 4 && (!x.q || x.q->sizes() == k.sizes()) && v.size(0) == k.size(0) &&
             v.size(1) == k.size(1),
         "expected q, k [B,T,H_q,K] and v [B,T,H_v,V]");
    const int64_t B = k.size(0), T = k.size(1), H_q = k.size(2), K = k.size(3), H_v = v.size(2), V = v.size(3);
    const int dtype = element(k.scalar_type());
    NEED(dtype >= 0 && v.scalar_type() == k.scalar_type() && (!x.q || x.q->scalar_type() == k.scalar_type()),
         "q, k, v must share one dtype, bfloat16 or float32");
    for (const at::Tensor *t : {x.g, x.beta})
        NEED(t->dim() == 3 && t->size(0) == B && t->size(1) == T && t->size(2) == H_v, "g and beta must be [B,T,H_v]");
    int64_t n_seq = B;
    if (x.cu) {
        NEED(B == 1 && x.cu->scalar_type() == at::kInt && x.cu->dim() == 1 && x.cu->numel() >= 1,
             "cu_seqlens must be int32 [N+1] with B == 1");
        if (!x.cu->is_cuda()) check_offsets(*x.cu, T);
        n_seq = x.cu->numel() - 1;
    }
    if (op != Op::STEP) check_parents(*x.parents, B, T, x.cu);
    NEED(states.scalar_type() == at::kFloat && states.dim() == 4 && states.size(1) == H_v && states.size(2) == K &&
             states.size(3) == V,
         "states must be float32 [n_slots,H_v,K,V]");
    check_slots(states, 0, "states");
    const int64_t n_slots = states.size(0);
    if (x.slots) {
        check_indices(*x.slots, n_seq, "slots", -1, n_slots);
        if (op != Op::TREE && !x.slots->is_cuda()) check_distinct(*x.slots);  // (trees only read)
    } else {
        NEED(n_slots >= n_seq, "states has ", n_slots, " slots for ", n_seq, " sequences");
    }
    if (op == Op::ACCEPT) check_accepted(*x.accepted, n_seq, T, x.cu);
    const at::Tensor *floating[] = {&k, &v, x.g, x.beta, &states, x.q};
    const NoGradient gradient;
    for (const at::Tensor *t : floating)
        if (t) gradient.check(*t);
    if (x.out) gradient.check(*x.out);  // (a backward through it would miss that it was written)
    const at::Device dev = states.device();
    NEED(dev.is_cuda(), "inputs must be on the GPU");
    for (const at::Tensor *t : floating) NEED(!t || t->device() == dev, "all tensors must be on one GPU");
    const c10::DeviceGuard guard(dev);
    if (op != Op::ACCEPT) {
        if (x.out) {
            o = *x.out;
            NEED(o.sizes() == v.sizes() && element(o.scalar_type()) >= 0 && o.is_contiguous() && aligned(o),
                 "out must be contiguous [B,T,H_v,V], bfloat16 or float32, 16-byte aligned");
            NEED(o.device() == dev, "all tensors must be on one GPU");
            for (const at::Tensor *t : floating) NEED(!overlap(o, *t), "out overlaps an input");
        } else {
            NEED(THPDtype_Check(x.output_dtype) &&
                     element(reinterpret_cast<THPDtype *>(x.output_dtype)->scalar_type) >= 0,
                 "output_dtype must be bfloat16 or float32");
            o = at::empty(v.sizes(), v.options().dtype(reinterpret_cast<THPDtype *>(x.output_dtype)->scalar_type));
        }
    }
    gdr_pool_args a = {};
    if (x.scale == Py_None) {
        a.scale = (float)(1.0 / std::sqrt((double)K));
    } else {
        a.scale = (float)PyFloat_AsDouble(x.scale);
        if (PyErr_Occurred()) return false;
    }
    Held held;
    const Rows kr = rows(k, held), vr = rows(v, held), qr = x.q ? rows(*x.q, held) : Rows{nullptr, 0, 0};
    a.B = B, a.T = T, a.H_q = H_q, a.H_v = H_v, a.K = K, a.V = V, a.n_seq = n_seq;
    a.n_slots = n_slots, a.slot_stride = states.stride(0);
    a.q = qr.data, a.q_row = qr.row, a.q_batch = qr.batch;
    a.k = kr.data, a.k_row = kr.row, a.k_batch = kr.batch;
    a.v = vr.data, a.v_row = vr.row, a.v_batch = vr.batch;
    a.dtype = dtype;
    a.out_dtype = o.defined() ? element(o.scalar_type()) : GDR_F32;
    a.g = floats(*x.g, held), a.beta = floats(*x.beta, held);
    a.cu_seqlens = indices(x.cu, dev, held), a.slots = indices(x.slots, dev, held);
    if (op != Op::STEP) a.parents = indices(x.parents, dev, held);
    if (op == Op::ACCEPT) a.accepted = indices(x.accepted, dev, held);
    a.states = static_cast<float *>(states.data_ptr());
    a.o = o.defined() ? o.data_ptr() : nullptr;
    if (op == Op::TREE) return launch(gdr_tree, "gdr_tree", a, dev, {x.out});
    if (op == Op::ACCEPT) return launch(gdr_tree_accept, "gdr_tree_accept", a, dev, {&states});
    return launch(gdr_step, "gdr_step", a, dev, {&states, x.out});
}

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return n == want;
}

// step(q, k, v, g, beta, states, scale, cu_seqlens, slots, output_dtype, out)
PyObject *step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 11)) return nullptr;
    const Call x = {&tensor(a[0], "q"), &tensor(a[1], "k"), &tensor(a[2], "v"), &tensor(a[3], "g"), &tensor(a[4], "beta"),
                    nullptr, nullptr, &tensor(a[5], "states"), optional_tensor(a[7], "cu_seqlens"),
                    optional_tensor(a[8], "slots"), optional_tensor(a[10], "out"), a[6], a[9]};
    at::Tensor o;
    return run(Op::STEP, x, o) ? THPVariable_Wrap(o) : nullptr;
    END_HANDLE_TH_ERRORS
}

// tree(q, k, v, g, beta, parents, states, scale, cu_seqlens, slots, output_dtype, out)
PyObject *tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 12)) return nullptr;
    const Call x = {&tensor(a[0], "q"), &tensor(a[1], "k"), &tensor(a[2], "v"), &tensor(a[3], "g"), &tensor(a[4], "beta"),
                    &tensor(a[5], "parents"), nullptr, &tensor(a[6], "states"), optional_tensor(a[8], "cu_seqlens"),
                    optional_tensor(a[9], "slots"), optional_tensor(a[11], "out"), a[7], a[10]};
    at::Tensor o;
    return run(Op::TREE, x, o) ? THPVariable_Wrap(o) : nullptr;
    END_HANDLE_TH_ERRORS
}

// accept(k, v, g, beta, parents, accepted, states, cu_seqlens, slots)
PyObject *accept(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 9)) return nullptr;
    const Call x = {nullptr, &tensor(a[0], "k"), &tensor(a[1], "v"), &tensor(a[2], "g"), &tensor(a[3], "beta"),
                    &tensor(a[4], "parents"), &tensor(a[5], "accepted"), &tensor(a[6], "states"),
                    optional_tensor(a[7], "cu_seqlens"), optional_tensor(a[8], "slots"), nullptr, Py_None, Py_None};
    at::Tensor o;
    if (!run(Op::ACCEPT, x, o)) return nullptr;
    return Py_NewRef(a[6]);
    END_HANDLE_TH_ERRORS
}

// one layer's pool [n_slots,H_v,K,V], or [layers,...] of them; the dimension of its slots
int check_pool(const at::Tensor &x, const char *name) {
    NEED(x.scalar_type() == at::kFloat && (x.dim() == 4 || x.dim() == 5), name,
         " must be float32 [n_slots,H_v,K,V] or [layers,n_slots,H_v,K,V]");
    if (x.dim() == 4) {
        check_slots(x, 0, name);
        return 0;
    }
    if (x.size(0) > 0) check_slots(x, 1, name);
    NEED(x.size(0) < 2 || (x.stride(0) % 4 == 0 && x.stride(0) >= x.size(2) * x.size(3) * x.size(4)), "a slot of ", name,
         " must be contiguous and 16-byte aligned");
    return 1;
}

// whether a state of one pool shares memory with one of the other; pools of equal strides may lie
// between each other's slots (those of unequal strides count as overlapping where their spans do)
bool pools_overlap(const at::Tensor &x, const at::Tensor &y, int at_slot) {
    if (!overlap(x, y)) return false;
    const int64_t nx = x.size(at_slot), ny = y.size(at_slot), layers = at_slot ? x.size(0) : 1;
    const int64_t state = 4 * x.size(at_slot + 1) * x.size(at_slot + 2) * x.size(at_slot + 3);
    const int64_t slot = 4 * (nx > 1 ? x : y).stride(at_slot), layer = layers > 1 ? 4 * x.stride(0) : 0;
    if ((nx > 1 && ny > 1 && x.stride(at_slot) != y.stride(at_slot)) || (layers > 1 && x.stride(0) != y.stride(0)))
        return true;
    const int64_t apart = (const char *)x.data_ptr() - (const char *)y.data_ptr();
    for (int64_t a = 1 - layers; a < layers; ++a) {
        // x's state s lies `at + (s - t) slot` bytes from y's t: s - t that bring them nearest
        const int64_t at = apart + a * layer, near = slot ? -at / slot : 0;
        for (int64_t b = near - 1; b <= near + 1; ++b) {
            const int64_t d = at + b * slot;
            if (b > -ny && b < nx && d > -state && d < state) return true;
        }
    }
    return false;
}

// copy(states, dst, src, source)
PyObject *copy(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (!count(n_args, 4)) return nullptr;
    const at::Tensor &states = tensor(a[0], "states"), &dst = tensor(a[1], "dst"), &src = tensor(a[2], "src"),
                     &source = a[3] == Py_None ? states : tensor(a[3], "source");
    const int at_slot = check_pool(states, "states");
    if (a[3] != Py_None) {
        const int other = check_pool(source, "source");
        NEED(other == at_slot && states.sizes().slice(at_slot + 1) == source.sizes().slice(at_slot + 1) &&
                 (at_slot == 0 || states.size(0) == source.size(0)),
             "states and source must hold states of one shape and as many layers");
        const bool same = source.data_ptr() == states.data_ptr() && source.sizes() == states.sizes() &&
                          source.strides() == states.strides();
        NEED(same || !pools_overlap(states, source, at_slot), "source overlaps states");
    }
    const int64_t n = dst.numel(), n_dst = states.size(at_slot), n_src = source.size(at_slot);
    NEED(n <= GDR_COPY_MAX, "at most ", GDR_COPY_MAX, " entries");
    check_indices(dst, n, "dst", -1, n_dst);
    check_indices(src, n, "src", -1, n_src);
    const NoGradient gradient;
    gradient.check(states);
    gradient.check(source);
    const at::Device dev = states.device();
    NEED(dev.is_cuda(), "inputs must be on the GPU");
    NEED(source.device() == dev, "all tensors must be on one GPU");
    const c10::DeviceGuard guard(dev);
    Held held;
    gdr_copy_args c = {};
    c.n = n, c.n_dst = n_dst, c.n_src = n_src;
    c.slot_bytes = 4 * states.size(at_slot + 1) * states.size(at_slot + 2) * states.size(at_slot + 3);
    c.dst_stride = 4 * states.stride(at_slot), c.src_stride = 4 * source.stride(at_slot);
    c.layers = at_slot ? states.size(0) : 1;
    c.dst_layer_stride = at_slot ? 4 * states.stride(0) : 0, c.src_layer_stride = at_slot ? 4 * source.stride(0) : 0;
    c.dst = indices(&dst, dev, held), c.src = indices(&src, dev, held);
    c.states = states.data_ptr(), c.source = source.data_ptr();
    if (!launch(gdr_copy_states, "gdr_copy_states", c, dev, {&states})) return nullptr;
    return Py_NewRef(a[0]);
    END_HANDLE_TH_ERRORS
}

// connect(GdrError, function from a device's index to its current stream's handle)
PyObject *connect(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 2)) return nullptr;
    // the argument blocks' layouts are compiled in here
    if (gdr_abi_version() != GDR_ABI_VERSION) {
        PyErr_Format(PyExc_ImportError, "libgdr ABI version %d, _gdr_torch is built for %d", gdr_abi_version(),
                     GDR_ABI_VERSION);
        return nullptr;
    }
    library_error = Py_NewRef(a[0]);
    current_stream = Py_NewRef(a[1]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"connect", (PyCFunction)(void (*)(void))connect, METH_FASTCALL, nullptr},
                         {"step", (PyCFunction)(void (*)(void))step, METH_FASTCALL, nullptr},
                         {"tree", (PyCFunction)(void (*)(void))tree, METH_FASTCALL, nullptr},
                         {"accept", (PyCFunction)(void (*)(void))accept, METH_FASTCALL, nullptr},
                         {"copy", (PyCFunction)(void (*)(void))copy, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdr_torch", "Checked calls of libgdr's operators on a pool of states.", -1,
                      methods};

}  // namespace

PyMODINIT_FUNC PyInit__gdr_torch(void) { return PyModule_Create(&module); }
