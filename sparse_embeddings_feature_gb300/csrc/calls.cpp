// The calls of the expert layer and of the layers around it from Python, in their usual layouts: the arguments' types and
// shapes are read from the tensors here, on the current stream, and the C entry point called.  A call whose arguments
// are anything else (strided rows, a wrong shape, tensors of another device than the current one, not a
// tensor) returns None: the binding in Python then takes it, with its own checks and messages.  Reading
// and checking eight tensors there, and handing 16 numbers over, takes 5 us of the host, more than the
// kernels of a small call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/ctr.h"

namespace {

struct Odd {};  // not the usual layout

thread_local int device = 0;  // the current one, where the call's kernels run

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Odd();
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous()) throw Odd();
  return t;
}

// Data of a dense tensor of the given type and shape; NULL for None where that is allowed.
template <typename T>
T* data(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape)) throw Odd();
  return (T*)t.data_ptr();
}

uint8_t* bytes(PyObject* o, std::initializer_list<int64_t> shape, bool optional = false) {
  return data<uint8_t>(o, at::kByte, shape, optional);
}
float* floats(PyObject* o, std::initializer_list<int64_t> shape, bool optional = false) {
  return data<float>(o, at::kFloat, shape, optional);
}
int32_t* ints(PyObject* o, std::initializer_list<int64_t> shape, bool optional = false) {
  return data<int32_t>(o, at::kInt, shape, optional);
}

// fp32 or bf16 values of the given number of dimensions.
struct Values {
  void* p;
  ctr_dtype type;
  at::ScalarType scalar;
  int64_t n[3];
  int64_t ld() const { return n[1] > 0 ? n[1] : 1; }  // of a matrix
};
Values values(PyObject* o, int dims) {
  const at::Tensor& t = tensor(o);
  Values v;
  v.scalar = t.scalar_type();
  if (t.dim() != dims || (v.scalar != at::kFloat && v.scalar != at::kBFloat16)) throw Odd();
  v.type = v.scalar == at::kFloat ? CTR_F32 : CTR_BF16;
  v.p = t.data_ptr();
  for (int i = 0; i < dims; ++i) v.n[i] = t.size(i);
  return v;
}

int64_t size(PyObject* o, int dims, int i) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != dims) throw Odd();
  return t.size(i);
}

int64_t number(PyObject* o) {
  const long long v = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
  if (v == -1) {
    PyErr_Clear();
    throw Odd();
  }
  return v;
}

// fp32 or bf16 values [rows, cols] of the given type; NULL for None.
void* like(PyObject* o, at::ScalarType type, int64_t rows, int64_t cols) {
  if (o == Py_None) return nullptr;
  const Values v = values(o, 2);
  if (v.n[0] != rows || v.n[1] != cols || v.scalar != type) throw Odd();
  return v.p;
}

float number_f32(PyObject* o) {
  if (!PyFloat_Check(o)) throw Odd();
  return (float)PyFloat_AS_DOUBLE(o);
}

struct Workspace {
  void* p;
  size_t n;
};
Workspace workspace(PyObject* o) {
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != at::kByte) throw Odd();
  return {t.data_ptr(), (size_t)t.numel()};
}

ctr_stream_t stream() { return (ctr_stream_t)c10::cuda::getCurrentCUDAStream().stream(); }
int64_t blocks(int64_t n) { return (n + 127) / 128; }

// Calls a C entry point without the interpreter's lock: a launch waits while the stream's queue is full, and other
// threads' Python is not to.  The arguments, which may refuse, are read before.
template <typename F, typename... A>
int free_of_lock(F f, A... args) {
  PyThreadState* state = PyEval_SaveThread();
  const int st = f(args...);
  PyEval_RestoreThread(state);
  return st;
}

// Runs a call and gives its status, or None.
template <int N, typename F>
PyObject* run(Py_ssize_t n, F&& call) {
  int st;
  if (n != N) Py_RETURN_NONE;
  try {
    device = c10::cuda::current_device();
    st = call();
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  return PyLong_FromLong(st);
}

#define CALL(name) PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n)

// scores, k, renormalize, expert, weight, slot, token, offsets, ws
CALL(expert_route) {
  return run<9>(n, [&] {
    const Values s = values(a[0], 2);
    const int64_t T = s.n[0], E = s.n[1], k = number(a[1]);
    const int renorm = PyObject_IsTrue(a[2]);
    if (k < 1 || k > E || renorm < 0) throw Odd();
    const Workspace w = workspace(a[8]);
    return free_of_lock(ctr_expert_route, s.p, s.type, T, (int32_t)E, s.ld(), (int32_t)k, renorm, ints(a[3], {T, k}),
                        floats(a[4], {T, k}), ints(a[5], {T, k}), ints(a[6], {T * k}), ints(a[7], {E + 1}), w.p, w.n,
                        stream());
  });
}

// dweight, scores, renormalize, expert, dscores, ws
CALL(expert_route_bwd) {
  return run<6>(n, [&] {
    const Values s = values(a[1], 2), d = values(a[4], 2);
    const int64_t T = s.n[0], E = s.n[1], k = size(a[3], 2, 1);
    const int renorm = PyObject_IsTrue(a[2]);
    if (d.n[0] != T || d.n[1] != E || d.scalar != s.scalar || k > E || renorm < 0) throw Odd();
    const Workspace w = workspace(a[5]);
    return free_of_lock(ctr_expert_route_bwd, floats(a[0], {T, k}), s.p, s.type, T, (int32_t)E, s.ld(), (int32_t)k,
                        renorm, ints(a[3], {T, k}), d.p, d.ld(), w.p, w.n, stream());
  });
}

// x, slot, token, out, ws
CALL(expert_dispatch) {
  return run<5>(n, [&] {
    const Values x = values(a[0], 2), o = values(a[3], 2);
    const int64_t T = x.n[0], d = x.n[1], k = size(a[1], 2, 1);
    if (o.n[0] != T * k || o.n[1] != d || o.scalar != x.scalar || d > INT32_MAX || k > INT32_MAX) throw Odd();
    const Workspace w = workspace(a[4]);
    return free_of_lock(ctr_expert_dispatch, x.p, x.type, T, (int32_t)d, x.ld(), (int32_t)k, ints(a[1], {T, k}),
                        ints(a[2], {T * k}), o.p, o.ld(), w.p, w.n, stream());
  });
}

// rows, slot, weight, y, ws
CALL(expert_combine) {
  return run<5>(n, [&] {
    const Values r = values(a[0], 2), y = values(a[3], 2);
    const int64_t T = y.n[0], d = y.n[1], k = size(a[1], 2, 1);
    if (r.n[0] != T * k || r.n[1] != d || r.scalar != y.scalar || d > INT32_MAX || k > INT32_MAX) throw Odd();
    const Workspace w = workspace(a[4]);
    return free_of_lock(ctr_expert_combine, r.p, r.type, T, (int32_t)d, r.ld(), (int32_t)k, ints(a[1], {T, k}),
                        floats(a[2], {T, k}, true), y.p, y.ld(), w.p, w.n, stream());
  });
}

// dy, rows, slot, weight, token, drows, dweight, ws
CALL(expert_combine_bwd) {
  return run<8>(n, [&] {
    const Values y = values(a[0], 2), r = values(a[1], 2), o = values(a[5], 2);
    const int64_t T = y.n[0], d = y.n[1], k = size(a[2], 2, 1);
    for (const Values& v : {r, o})
      if (v.n[0] != T * k || v.n[1] != d || v.scalar != y.scalar) throw Odd();
    if (d > INT32_MAX || k > INT32_MAX) throw Odd();
    const Workspace w = workspace(a[7]);
    return free_of_lock(ctr_expert_combine_bwd, y.p, y.type, T, (int32_t)d, y.ld(), (int32_t)k, r.p, r.ld(),
                        ints(a[2], {T, k}), floats(a[3], {T, k}), ints(a[4], {T * k}), o.p, o.ld(),
                        floats(a[6], {T, k}), w.p, w.n, stream());
  });
}

// x, q, scale, ws, row_index
CALL(fp8_quantize_rows) {
  return run<5>(n, [&] {
    const Values x = values(a[0], 2);
    const int64_t cols = x.n[1], rows = size(a[1], 2, 0), kb = blocks(cols);
    if (a[4] == Py_None && rows > x.n[0]) throw Odd();
    const Workspace w = workspace(a[3]);
    return free_of_lock(ctr_fp8_quantize_rows, x.p, x.type, x.n[0], rows, cols, x.ld(), ints(a[4], {rows}, true),
                        bytes(a[1], {rows, kb * 128}), floats(a[2], {kb, rows}), rows > 0 ? rows : 1, w.p, w.n,
                        stream());
  });
}

// x, offsets, q, scale, qc, scale_c, cols_by_block, ws, row_index
CALL(fp8_quantize_rows_cols) {
  return run<9>(n, [&] {
    const Values x = values(a[0], 2);
    const int64_t cols = x.n[1], rows = size(a[2], 2, 0), kb = blocks(cols), groups = size(a[1], 1, 0) - 1;
    const int64_t by_block = number(a[6]);
    if ((a[8] == Py_None && rows > x.n[0]) || groups < 1 || groups > INT32_MAX || by_block < 0 || by_block > 1)
      throw Odd();
    const int64_t padded = ctr_fp8_padded_rows(rows, (int32_t)groups);
    float* sc = by_block ? floats(a[5], {kb, padded / 128}) : floats(a[5], {padded / 128, cols});
    const Workspace w = workspace(a[7]);
    return free_of_lock(ctr_fp8_quantize_rows_cols, x.p, x.type, x.n[0], rows, cols, x.ld(), ints(a[8], {rows}, true),
                        ints(a[1], {groups + 1}), (int32_t)groups, (int)by_block, bytes(a[2], {rows, kb * 128}),
                        floats(a[3], {kb, rows}), rows > 0 ? rows : 1, bytes(a[4], {cols, padded}), sc, w.p, w.n,
                        stream());
  });
}

// w, q, scale, ws, qt, scale_t
CALL(fp8_quantize_blocks) {
  return run<6>(n, [&] {
    const Values v = values(a[0], 3);
    const int64_t G = v.n[0], r = v.n[1], k = v.n[2], nb = blocks(r), kb = blocks(k);
    if (G > INT32_MAX || (a[4] == Py_None) != (a[5] == Py_None)) throw Odd();
    const Workspace w = workspace(a[3]);
    return free_of_lock(ctr_fp8_quantize_blocks, v.p, v.type, (int32_t)G, r, k, bytes(a[1], {G, r, kb * 128}),
                        floats(a[2], {G, nb, kb}), bytes(a[4], {G, k, nb * 128}, true),
                        floats(a[5], {G, kb, nb}, true), w.p, w.n, stream());
  });
}

// a, a_scale, b, b_scale, offsets, out, ws
CALL(fp8_matmul) {
  return run<7>(n, [&] {
    const Values o = values(a[5], 2);
    const int64_t rows = o.n[0], cols = o.n[1], G = size(a[2], 3, 0), kp = size(a[2], 3, 2), kb = kp / 128;
    if (kp < 128 || kp % 128 || G > INT32_MAX) throw Odd();
    const Workspace w = workspace(a[6]);
    return free_of_lock(ctr_fp8_matmul, bytes(a[0], {rows, kp}), floats(a[1], {kb, rows}), rows > 0 ? rows : 1,
                        bytes(a[2], {G, cols, kp}), floats(a[3], {G, blocks(cols), kb}), ints(a[4], {G + 1}, true),
                        rows, (int32_t)G, cols, kp, o.p, o.type, o.ld(), w.p, w.n, stream());
  });
}

// d, d_scale, x, x_scale, offsets, out, ws, rows (None: the most that have the codes' padding)
CALL(fp8_matmul_wgrad) {
  return run<8>(n, [&] {
    const Values o = values(a[5], 3);
    const int64_t G = o.n[0], r = o.n[1], k = o.n[2], padded = size(a[0], 2, 1), tiles = padded / 128;
    const int64_t most = (tiles + 1) * 128 - 1 - 127 * G;  // rows that have this padding
    const int64_t rows = a[7] != Py_None ? number(a[7]) : most > tiles ? most : tiles;
    if (G < 1 || G > INT32_MAX || rows < 0 || ctr_fp8_padded_rows(rows, (int32_t)G) != padded) throw Odd();
    const Workspace w = workspace(a[6]);
    return free_of_lock(ctr_fp8_matmul_wgrad, bytes(a[0], {r, padded}), floats(a[1], {padded / 128, r}),
                        bytes(a[2], {k, padded}), floats(a[3], {blocks(k), padded / 128}), ints(a[4], {G + 1}), rows,
                        (int32_t)G, r, k, o.p, o.type, w.p, w.n, stream());
  });
}

// addresses of grads, outs (or None), dtypes, counts; number of tensors, their device (or None), max_norm, norm, ws
CALL(clip_grads) {
  return run<9>(n, [&] {
    const int64_t grads = number(a[0]), outs = a[1] == Py_None ? 0 : number(a[1]), types = number(a[2]);
    const int64_t counts = number(a[3]), tensors = number(a[4]);
    if (!PyFloat_Check(a[6]) || tensors > INT32_MAX || (a[5] != Py_None && number(a[5]) != device)) throw Odd();
    const Workspace w = workspace(a[8]);
    return free_of_lock(ctr_clip_grads, (const void* const*)grads, (void* const*)outs, (const int32_t*)types,
                        (const int64_t*)counts, (int32_t)tensors, (float)PyFloat_AS_DOUBLE(a[6]), floats(a[7], {1}),
                        w.p, w.n, stream());
  });
}

// scores, k, score, bias, groups, group_k, renormalize, factor, expert, weight, slot, token, offsets, ws
CALL(expert_route_balanced) {
  return run<14>(n, [&] {
    const Values s = values(a[0], 2);
    const int64_t T = s.n[0], E = s.n[1], k = number(a[1]), score = number(a[2]), groups = number(a[4]), kept = number(a[5]);
    const int renorm = PyObject_IsTrue(a[6]);
    if (k < 1 || k > E || renorm < 0 || E > INT32_MAX || score < 0 || score > 1 || groups < 1 || groups > E || kept < 1 ||
        kept > groups)
      throw Odd();
    const Workspace w = workspace(a[13]);
    return free_of_lock(ctr_expert_route_balanced, s.p, s.type, T, (int32_t)E, s.ld(), (int32_t)k, (int)score,
                        floats(a[3], {E}, true), (int32_t)groups, (int32_t)kept, renorm, number_f32(a[7]), ints(a[8], {T, k}),
                        floats(a[9], {T, k}), ints(a[10], {T, k}), ints(a[11], {T * k}), ints(a[12], {E + 1}), w.p, w.n,
                        stream());
  });
}

// dweight, scores, score, renormalize, factor, expert, dscores, ws
CALL(expert_route_balanced_bwd) {
  return run<8>(n, [&] {
    const Values s = values(a[1], 2), d = values(a[6], 2);
    const int64_t T = s.n[0], E = s.n[1], score = number(a[2]), k = size(a[5], 2, 1);
    const int renorm = PyObject_IsTrue(a[3]);
    if (d.n[0] != T || d.n[1] != E || d.scalar != s.scalar || k > E || renorm < 0 || score < 0 || score > 1) throw Odd();
    const Workspace w = workspace(a[7]);
    return free_of_lock(ctr_expert_route_balanced_bwd, floats(a[0], {T, k}), s.p, s.type, T, (int32_t)E, s.ld(), (int32_t)k,
                        (int)score, renorm, number_f32(a[4]), ints(a[5], {T, k}), d.p, d.ld(), w.p, w.n, stream());
  });
}

// x, w, bias, act, residual, y, pre, ws
CALL(dense) {
  return run<8>(n, [&] {
    const Values x = values(a[0], 2), w = values(a[1], 2), y = values(a[5], 2);
    const int64_t rows = x.n[0], k = x.n[1], cols = w.n[0], act = number(a[3]);
    if (w.n[1] != k || w.scalar != x.scalar || y.n[0] != rows || y.n[1] != cols || y.scalar != x.scalar || act > INT32_MAX)
      throw Odd();
    const Workspace room = workspace(a[7]);
    return free_of_lock(ctr_dense, x.p, x.type, rows, k, x.ld(), w.p, cols, w.ld(), data<void>(a[2], x.scalar, {cols}, true),
                        (int)act, like(a[4], x.scalar, rows, cols), y.ld(), y.p, y.ld(), like(a[6], x.scalar, rows, cols),
                        y.ld(), room.p, room.n, stream());
  });
}

// dy, x, w, pre, act, dx, dw, dbias, ws
CALL(dense_bwd) {
  return run<9>(n, [&] {
    const Values y = values(a[0], 2), x = values(a[1], 2);
    const int64_t rows = y.n[0], cols = y.n[1], k = x.n[1], act = number(a[4]);
    if (x.n[0] != rows || x.scalar != y.scalar || a[2] == Py_None || act > INT32_MAX || (act != 0 && a[3] == Py_None))
      throw Odd();
    PyObject* some = a[6] != Py_None ? a[6] : a[7];
    const at::ScalarType grad = some != Py_None ? tensor(some).scalar_type() : y.scalar;
    if (grad != at::kFloat && grad != y.scalar) throw Odd();
    const Workspace room = workspace(a[8]);
    return free_of_lock(ctr_dense_bwd, y.p, y.type, rows, cols, y.ld(), x.p, k, x.ld(), like(a[2], y.scalar, cols, k),
                        x.ld(), like(a[3], y.scalar, rows, cols), y.ld(), (int)act, like(a[5], y.scalar, rows, k), x.ld(),
                        grad == at::kFloat ? CTR_F32 : CTR_BF16, like(a[6], grad, cols, k), x.ld(),
                        data<void>(a[7], grad, {cols}, true), room.p, room.n, stream());
  });
}

// x, residual, gamma, eps, s, y, q, scale, ws
CALL(rms_norm) {
  return run<9>(n, [&] {
    const Values x = values(a[0], 2);
    const int64_t rows = x.n[0], d = x.n[1], kb = blocks(d), ld = x.ld();
    if (d > INT32_MAX || (a[6] == Py_None) != (a[7] == Py_None)) throw Odd();
    const Workspace w = workspace(a[8]);
    return free_of_lock(ctr_rms_norm, x.p, x.type, rows, (int32_t)d, ld, like(a[1], x.scalar, rows, d), ld,
                        floats(a[2], {d}, true), number_f32(a[3]), like(a[4], x.scalar, rows, d), ld,
                        like(a[5], x.scalar, rows, d), ld, bytes(a[6], {rows, kb * 128}, true),
                        floats(a[7], {kb, rows}, true), rows > 0 ? rows : 1, w.p, w.n, stream());
  });
}

// dy, ds, s, gamma, eps, dx, dgamma, ws
CALL(rms_norm_bwd) {
  return run<8>(n, [&] {
    const Values y = values(a[0], 2);
    const int64_t rows = y.n[0], d = y.n[1], ld = y.ld();
    if (d > INT32_MAX || a[2] == Py_None || a[5] == Py_None) throw Odd();
    const Workspace w = workspace(a[7]);
    return free_of_lock(ctr_rms_norm_bwd, y.p, y.type, rows, (int32_t)d, ld, like(a[1], y.scalar, rows, d), ld,
                        like(a[2], y.scalar, rows, d), ld, floats(a[3], {d}, true), number_f32(a[4]),
                        like(a[5], y.scalar, rows, d), ld, floats(a[6], {d}, true), w.p, w.n, stream());
  });
}

#define ENTRY(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(expert_route),          ENTRY(expert_route_bwd),   ENTRY(expert_dispatch),
                         ENTRY(expert_combine),        ENTRY(expert_combine_bwd), ENTRY(fp8_quantize_rows),
                         ENTRY(fp8_quantize_rows_cols), ENTRY(fp8_quantize_blocks), ENTRY(fp8_matmul),
                         ENTRY(fp8_matmul_wgrad),      ENTRY(clip_grads),
                         ENTRY(dense),                 ENTRY(dense_bwd),          ENTRY(rms_norm),
                         ENTRY(rms_norm_bwd),          ENTRY(expert_route_balanced), ENTRY(expert_route_balanced_bwd),
                               {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ctr_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ctr_calls(void) { return PyModule_Create(&module); }
