// Python entry points of the speculative-decoding operators and of those around a
// step's attention over the C ABI.
//
// A step of these operators takes the GPU a few microseconds, while marshalling
// ten tensors through ctypes took the host 20 to 40: this module reads the
// tensors, allocates the outputs and calls the library from C++.  It computes
// nothing; libfw_attn.so does not depend on it, and every other entry point
// stays in _binding.py, which hands over the library's functions once.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cstdarg>

#include "fw_attn.h"

namespace {

decltype(&fw_paged_decode_tree) g_tree;
decltype(&fw_paged_decode_tree_workspace_size) g_tree_workspace;
decltype(&fw_tree_mask) g_mask;
decltype(&fw_build_page_tables) g_tables;
decltype(&fw_kv_commit) g_commit;
decltype(&fw_verify_drafts) g_verify;
decltype(&fw_paged_prefill) g_prefill;
decltype(&fw_paged_prefill_workspace_size) g_prefill_workspace;
decltype(&fw_qk_norm_rope) g_norm_rope;
decltype(&fw_qk_norm_rope_append) g_norm_rope_append;
PyObject *g_check;                     // raises FwError for a status

[[noreturn]] void raise(PyObject *type, const char *format, ...) {
    va_list ap;
    va_start(ap, format);
    PyErr_FormatV(type, format, ap);
    va_end(ap);
    python_error e;
    e.persist();
    throw e;
}

// The tensors of one call: views for the C ABI, and the one device they share.
struct Args {
    int device = -1;
    std::array<fw_tensor_t, 16> view;
    int count = 0;

    // The tensor behind a Python object; None gives an undefined one.
    static at::Tensor take(PyObject *o, const char *name) {
        if (o == Py_None) return {};
        if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
        return THPVariable_Unpack(o);
    }
    void place(const at::Tensor &t) {
        if (!t.defined()) return;
        if (!t.is_cuda()) raise(PyExc_ValueError, "the tensors must be on a CUDA device");
        if (device < 0) device = t.get_device();
        else if (device != t.get_device()) raise(PyExc_ValueError, "the tensors must be on one device");
    }
    fw_tensor_t *add(const at::Tensor &t) {
        if (!t.defined()) return nullptr;
        fw_tensor_t &v = view[count++];
        switch (t.scalar_type()) {
            case at::kBFloat16: v.dtype = FW_BF16; break;
            case at::kFloat: v.dtype = FW_F32; break;
            case at::kInt: v.dtype = FW_I32; break;
            case at::kFloat8_e4m3fn: v.dtype = FW_FP8_E4M3; break;
            default: raise(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
        }
        if (t.dim() > 5) raise(PyExc_ValueError, "at most 5 dimensions");
        v.data = t.numel() > 0 ? t.data_ptr() : nullptr;
        v.ndim = (int32_t)t.dim();
        for (int i = 0; i < v.ndim; ++i) {
            v.shape[i] = t.size(i);
            v.stride[i] = t.stride(i);
        }
        return &v;
    }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int device) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
}

// Contiguous int32 outputs of one call, cut from one allocation: taking a buffer
// from torch's allocator costs the host as much as a quarter of a launch, and
// these calls are as short as that.
struct Outputs {
    at::Tensor buffer;
    int64_t used = 0;

    static int64_t room(int64_t n) { return (n + 63) / 64 * 64; }      // 256-byte pieces
    Outputs(int64_t total, int device) {
        if (total > 0) buffer = empty({total}, at::kInt, device);
    }
    at::Tensor cut(at::IntArrayRef shape) {
        int64_t n = 1;
        for (const int64_t s : shape) n *= s;
        auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(), buffer.dtype());
        impl->set_storage_offset(used);
        impl->set_sizes_contiguous(shape);
        used += room(n);
        return at::Tensor(std::move(impl));
    }
};

// The current stream of the call's device, which is current while this lives.
struct Where {
    c10::cuda::CUDAGuard guard;
    explicit Where(int device) : guard((c10::DeviceIndex)device) {}
    fw_stream_t stream() const {
        return reinterpret_cast<fw_stream_t>(c10::cuda::getCurrentCUDAStream(guard.current_device().index()).stream());
    }
};

void need(const at::Tensor &t, const char *name) {
    if (!t.defined()) raise(PyExc_TypeError, "%s is required", name);
}

bool failed(fw_status_t st) {
    if (st == FW_OK) return false;
    PyObject *r = PyObject_CallFunction(g_check, "i", (int)st);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "call failed");
    return true;
}

bool arity(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return false;
}

bool number(PyObject *o, double *v) {
    *v = PyFloat_AsDouble(o);
    return !(*v == -1.0 && PyErr_Occurred());
}

bool whole(PyObject *o, long long *v) {
    PyObject *i = PyNumber_Index(o);
    if (!i) return false;
    *v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    return !(*v == -1 && PyErr_Occurred());
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
    return Py_BuildValue("NN", THPVariable_Wrap(a), b.defined() ? THPVariable_Wrap(b) : Py_NewRef(Py_None));
}

// (q, k_cache, v_cache, block_table, seq_lens, tree_mask, draft_lens, scale,
//  k_scale, v_scale, out, lse, return_lse, workspace)
PyObject *paged_decode_tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 14)) return nullptr;
    double scale, ks, vs;
    if (!number(a[7], &scale) || !number(a[8], &ks) || !number(a[9], &vs)) return nullptr;
    const char *names[7] = {"q", "k_cache", "v_cache", "block_table", "seq_lens", "tree_mask", "draft_lens"};
    at::Tensor t[7];
    Args args;
    for (int i = 0; i < 7; ++i) {
        t[i] = Args::take(a[i], names[i]);
        if (i < 6) need(t[i], names[i]);
        args.place(t[i]);
    }
    at::Tensor out = Args::take(a[10], "out"), lse = Args::take(a[11], "lse"), ws = Args::take(a[13], "workspace");
    args.place(out);
    args.place(lse);
    args.place(ws);
    if (t[0].dim() != 4) raise(PyExc_ValueError, "q must be [B, T, Hq, D]");
    const bool want_lse = PyObject_IsTrue(a[12]);
    Where where(args.device);
    if (!out.defined()) out = empty(t[0].sizes(), at::kBFloat16, args.device);
    if (!lse.defined() && want_lse) lse = empty(t[0].sizes().slice(0, 3), at::kFloat, args.device);
    if (!ws.defined()) {
        size_t bytes = 0;
        if (failed(g_tree_workspace((int32_t)t[0].size(3), &bytes))) return nullptr;
        ws = empty({(int64_t)bytes}, at::kByte, args.device);
    } else if (!ws.is_contiguous()) {
        raise(PyExc_ValueError, "workspace must be contiguous");
    }
    fw_tensor_t *v[7];
    for (int i = 0; i < 7; ++i) v[i] = args.add(t[i]);
    fw_tensor_t *vo = args.add(out), *vl = args.add(lse);
    // NULL would mean the library's own buffer, which calls on several streams share: a
    // caller's empty tensor is a workspace of no bytes (at an address that is not read).
    void *room = ws.nbytes() > 0 ? ws.data_ptr() : reinterpret_cast<void *>(256);
    if (failed(g_tree(v[0], v[1], v[2], v[3], v[4], v[5], v[6], (float)scale, (float)ks, (float)vs, vo, vl, room,
                      ws.nbytes(), where.stream())))
        return nullptr;
    return pair(out, lse);
    END_HANDLE_TH_ERRORS
}

// (parents, draft_lens, mask, depths)
PyObject *tree_mask(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 4)) return nullptr;
    at::Tensor par = Args::take(a[0], "parents"), dl = Args::take(a[1], "draft_lens");
    at::Tensor mask = Args::take(a[2], "mask"), depths = Args::take(a[3], "depths");
    need(par, "parents");
    Args args;
    args.place(par);
    args.place(dl);
    args.place(mask);
    args.place(depths);
    if (par.dim() != 2) raise(PyExc_ValueError, "parents must be [B, T]");
    Where where(args.device);
    const int64_t B = par.size(0), T = par.size(1);
    const int64_t W = (T + 31) / 32;
    Outputs outs((mask.defined() ? 0 : Outputs::room(B * T * W)) + (depths.defined() ? 0 : Outputs::room(B * T)), args.device);
    if (!mask.defined()) mask = outs.buffer.defined() ? outs.cut({B, T, W}) : empty({B, T, W}, at::kInt, args.device);
    if (!depths.defined()) depths = outs.buffer.defined() ? outs.cut({B, T}) : empty({B, T}, at::kInt, args.device);
    fw_tensor_t *v0 = args.add(par), *v1 = args.add(dl), *v2 = args.add(mask), *v3 = args.add(depths);
    if (failed(g_mask(v0, v1, v2, v3, where.stream()))) return nullptr;
    return pair(mask, depths);
    END_HANDLE_TH_ERRORS
}

// (seq_lens, new_lens, held, free_queue, free_range, page_size, block_table,
//  slot_mapping, cu_new, held_out, range_out)
PyObject *build_page_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 11)) return nullptr;
    long long page_size;
    if (!whole(a[5], &page_size)) return nullptr;
    const char *names[11] = {"seq_lens", "new_lens", "held", "free_queue", "free_range", "", "block_table",
                             "slot_mapping", "cu_new", "held_out", "range_out"};
    at::Tensor t[11];
    Args args;
    for (int i = 0; i < 11; ++i) {
        if (i == 5) continue;
        t[i] = Args::take(a[i], names[i]);
        if (i < 8) need(t[i], names[i]);
        args.place(t[i]);
    }
    Where where(args.device);
    const int64_t B = t[0].numel();
    int64_t total = 0;
    const int64_t sizes[3] = {B + 1, B, 2};
    for (int i = 0; i < 3; ++i)
        if (!t[8 + i].defined()) total += Outputs::room(sizes[i]) + 64;
    Outputs outs(total, args.device);
    for (int i = 0; i < 3; ++i)
        if (!t[8 + i].defined()) t[8 + i] = outs.cut({sizes[i]});
    fw_tensor_t *v[11];
    for (int i = 0; i < 11; ++i) v[i] = i == 5 ? nullptr : args.add(t[i]);
    if (failed(g_tables(v[0], v[1], v[2], v[3], v[4], page_size, v[6], v[7], v[8], v[9], v[10], where.stream())))
        return nullptr;
    return Py_BuildValue("NNN", THPVariable_Wrap(t[8]), THPVariable_Wrap(t[9]), THPVariable_Wrap(t[10]));
    END_HANDLE_TH_ERRORS
}

// (path, path_lens, base_lens, block_table, k_cache, v_cache, num_layers, new_lens)
PyObject *kv_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 8)) return nullptr;
    long long layers;
    if (!whole(a[6], &layers)) return nullptr;
    const char *names[8] = {"path", "path_lens", "base_lens", "block_table", "k_cache", "v_cache", "", "new_lens"};
    at::Tensor t[8];
    Args args;
    for (int i = 0; i < 8; ++i) {
        if (i == 6) continue;
        t[i] = Args::take(a[i], names[i]);
        if (i < 5) need(t[i], names[i]);
        args.place(t[i]);
    }
    Where where(args.device);
    if (!t[7].defined()) t[7] = empty({t[1].numel()}, at::kInt, args.device);
    fw_tensor_t *v[8];
    for (int i = 0; i < 8; ++i) v[i] = i == 6 ? nullptr : args.add(t[i]);
    if (failed(g_commit(v[0], v[1], v[2], v[3], layers, v[4], v[5], v[7], where.stream()))) return nullptr;
    return THPVariable_Wrap(t[7]);
    END_HANDLE_TH_ERRORS
}

// (tokens, parents, target_probs, uniforms, draft_probs, draft_lens, max_path, path,
//  path_lens, next_tokens)
PyObject *verify_drafts(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 10)) return nullptr;
    const char *names[10] = {"tokens", "parents", "target_probs", "uniforms", "draft_probs", "draft_lens", "", "path",
                             "path_lens", "next_tokens"};
    at::Tensor t[10];
    Args args;
    for (int i = 0; i < 10; ++i) {
        if (i == 6) continue;
        t[i] = Args::take(a[i], names[i]);
        if (i < 4) need(t[i], names[i]);
        args.place(t[i]);
    }
    if (t[0].dim() != 2) raise(PyExc_ValueError, "tokens must be [B, T]");
    const int64_t B = t[0].size(0);
    long long most = t[0].size(1);
    if (a[6] != Py_None && !whole(a[6], &most)) return nullptr;
    if (!t[7].defined() && (most < 1 || most > 256)) raise(PyExc_ValueError, "max_path must be 1 to 256");
    // A given path's width is how many are accepted at most.
    if (t[7].defined() && a[6] != Py_None && (t[7].dim() != 2 || t[7].size(1) != most))
        raise(PyExc_ValueError, "path must be [B, max_path] where both are given");
    Where where(args.device);
    const int64_t sizes[3] = {B * (int64_t)most, B, B};
    int64_t total = 0;
    for (int i = 0; i < 3; ++i)
        if (!t[7 + i].defined()) total += Outputs::room(sizes[i]) + 64;
    Outputs outs(total, args.device);
    if (!t[7].defined()) t[7] = outs.cut({B, (int64_t)most});
    for (int i = 1; i < 3; ++i)
        if (!t[7 + i].defined()) t[7 + i] = outs.cut({B});
    fw_tensor_t *v[10];
    for (int i = 0; i < 10; ++i) v[i] = i == 6 ? nullptr : args.add(t[i]);
    if (failed(g_verify(v[0], v[1], v[5], v[2], v[4], v[3], v[7], v[8], v[9], where.stream()))) return nullptr;
    return Py_BuildValue("NNN", THPVariable_Wrap(t[7]), THPVariable_Wrap(t[8]), THPVariable_Wrap(t[9]));
    END_HANDLE_TH_ERRORS
}

// (q, k, positions, inv_freq, q_weight, k_weight, eps, axis_map, interleaved, q_out, k_out)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 11)) return nullptr;
    double eps;
    if (!number(a[6], &eps)) return nullptr;
    const int interleaved = PyObject_IsTrue(a[8]);
    if (interleaved < 0) return nullptr;
    const char *names[11] = {"q", "k", "positions", "inv_freq", "q_weight", "k_weight", "", "axis_map", "", "q_out", "k_out"};
    at::Tensor t[11];
    Args args;
    for (int i = 0; i < 11; ++i) {
        if (i == 6 || i == 8) continue;
        t[i] = Args::take(a[i], names[i]);
        if (i < 4) need(t[i], names[i]);
        args.place(t[i]);
    }
    Where where(args.device);
    for (int i = 0; i < 2; ++i)
        if (!t[9 + i].defined()) t[9 + i] = empty(t[i].sizes(), at::kBFloat16, args.device);
    fw_tensor_t *v[11];
    for (int i = 0; i < 11; ++i) v[i] = i == 6 || i == 8 ? nullptr : args.add(t[i]);
    if (failed(g_norm_rope(v[0], v[1], v[4], v[5], (float)eps, v[3], v[2], v[7], interleaved, v[9], v[10], where.stream())))
        return nullptr;
    return pair(t[9], t[10]);
    END_HANDLE_TH_ERRORS
}

// (q, k, v, positions, inv_freq, slot_mapping, layer_base_rows, k_cache, v_cache,
//  q_weight, k_weight, eps, axis_map, interleaved, k_scale, v_scale, q_out)
PyObject *qk_norm_rope_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 17)) return nullptr;
    double eps, ks, vs;
    long long base;
    if (!whole(a[6], &base) || !number(a[11], &eps) || !number(a[14], &ks) || !number(a[15], &vs)) return nullptr;
    const int interleaved = PyObject_IsTrue(a[13]);
    if (interleaved < 0) return nullptr;
    const char *names[17] = {"q", "k", "v", "positions", "inv_freq", "slot_mapping", "", "k_cache", "v_cache", "q_weight",
                             "k_weight", "", "axis_map", "", "", "", "q_out"};
    at::Tensor t[17];
    Args args;
    for (int i = 0; i < 17; ++i) {
        if (!names[i][0]) continue;
        t[i] = Args::take(a[i], names[i]);
        if (i < 8 && i != 2) need(t[i], names[i]);
        args.place(t[i]);
    }
    Where where(args.device);
    if (!t[16].defined()) t[16] = empty(t[0].sizes(), at::kBFloat16, args.device);
    fw_tensor_t *v[17];
    for (int i = 0; i < 17; ++i) v[i] = names[i][0] ? args.add(t[i]) : nullptr;
    if (failed(g_norm_rope_append(v[0], v[1], v[2], v[9], v[10], (float)eps, v[4], v[3], v[12], interleaved, v[5], base,
                                  v[16], v[7], v[8], (float)ks, (float)vs, where.stream())))
        return nullptr;
    return THPVariable_Wrap(t[16]);
    END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens, scale, causal,
//  window_left, k_scale, v_scale, out, lse, return_lse, workspace)
PyObject *paged_prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 15)) return nullptr;
    double scale, ks, vs;
    long long window;
    if (!number(a[6], &scale) || !whole(a[8], &window) || !number(a[9], &ks) || !number(a[10], &vs)) return nullptr;
    const int causal = PyObject_IsTrue(a[7]), want_lse = PyObject_IsTrue(a[13]);
    if (causal < 0 || want_lse < 0) return nullptr;
    if (window > INT32_MAX) window = INT32_MAX;        // no key is that far
    if (window < -1) raise(PyExc_ValueError, "window_left must be -1 or more");
    const char *names[6] = {"q", "k_cache", "v_cache", "block_table", "cu_seqlens_q", "seq_lens"};
    at::Tensor t[6];
    Args args;
    for (int i = 0; i < 6; ++i) {
        t[i] = Args::take(a[i], names[i]);
        need(t[i], names[i]);
        args.place(t[i]);
    }
    at::Tensor out = Args::take(a[11], "out"), lse = Args::take(a[12], "lse"), ws = Args::take(a[14], "workspace");
    args.place(out);
    args.place(lse);
    args.place(ws);
    if (t[0].dim() != 3) raise(PyExc_ValueError, "q must be [total_q, Hq, D]");
    Where where(args.device);
    if (!out.defined()) out = empty(t[0].sizes(), at::kBFloat16, args.device);
    if (!lse.defined() && want_lse) lse = empty(t[0].sizes().slice(0, 2), at::kFloat, args.device);
    if (!ws.defined()) {
        size_t bytes = 0;
        if (failed(g_prefill_workspace((int32_t)t[0].size(2), &bytes))) return nullptr;
        ws = empty({(int64_t)bytes}, at::kByte, args.device);
    } else if (!ws.is_contiguous()) {
        raise(PyExc_ValueError, "workspace must be contiguous");
    }
    fw_tensor_t *v[6];
    for (int i = 0; i < 6; ++i) v[i] = args.add(t[i]);
    fw_tensor_t *vo = args.add(out), *vl = args.add(lse);
    // As in paged_decode_tree: a caller's empty tensor is a workspace of no bytes.
    void *room = ws.nbytes() > 0 ? ws.data_ptr() : reinterpret_cast<void *>(256);
    if (failed(g_prefill(v[0], v[1], v[2], v[3], v[4], v[5], (float)scale, (float)ks, (float)vs, causal, (int32_t)window, vo,
                         vl, room, ws.nbytes(), where.stream())))
        return nullptr;
    return pair(out, lse);
    END_HANDLE_TH_ERRORS
}

// (addresses of the C entry points, the status check)
PyObject *connect(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr int kEntries = 10;
    if (!arity(n, kEntries + 1)) return nullptr;
    void *f[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a NULL entry point");
            return nullptr;
        }
    }
    g_tree = reinterpret_cast<decltype(g_tree)>(f[0]);
    g_tree_workspace = reinterpret_cast<decltype(g_tree_workspace)>(f[1]);
    g_mask = reinterpret_cast<decltype(g_mask)>(f[2]);
    g_tables = reinterpret_cast<decltype(g_tables)>(f[3]);
    g_commit = reinterpret_cast<decltype(g_commit)>(f[4]);
    g_verify = reinterpret_cast<decltype(g_verify)>(f[5]);
    g_norm_rope = reinterpret_cast<decltype(g_norm_rope)>(f[6]);
    g_norm_rope_append = reinterpret_cast<decltype(g_norm_rope_append)>(f[7]);
    g_prefill = reinterpret_cast<decltype(g_prefill)>(f[8]);
    g_prefill_workspace = reinterpret_cast<decltype(g_prefill_workspace)>(f[9]);
    Py_XSETREF(g_check, Py_NewRef(a[kEntries]));
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"connect", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(connect)), METH_FASTCALL, nullptr},
    {"paged_decode_tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(paged_decode_tree)), METH_FASTCALL, nullptr},
    {"tree_mask", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(tree_mask)), METH_FASTCALL, nullptr},
    {"build_page_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(build_page_tables)), METH_FASTCALL, nullptr},
    {"kv_commit", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv_commit)), METH_FASTCALL, nullptr},
    {"paged_prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(paged_prefill)), METH_FASTCALL, nullptr},
    {"verify_drafts", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(verify_drafts)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"qk_norm_rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(qk_norm_rope_append)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fw_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fw_fast(void) { return PyModule_Create(&module); }
