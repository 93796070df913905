// Native marshalling of the long-cache calls: torch tensors in, libdec entry
// points out.  These calls take a few microseconds on the GPU, and checking
// seven tensors in Python with a ctypes call behind takes 10; here it is well
// under one.  Same rules as the Python side: wrong dtypes raise TypeError,
// layouts ValueError, everything else DecError with the library's codes.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "libdec.h"

namespace {

PyObject* g_dec_error = nullptr;  // the DecError class

struct Failure {
  PyObject* type;  // null: DecError(code, text)
  int code;
  std::string text;
};

[[noreturn]] void refuse(const std::string& text) { throw Failure{nullptr, DEC_EINVAL, text}; }
void expect(bool ok, const std::string& text) {
  if (!ok) refuse(text);
}

std::string str(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << ")";
  return o.str();
}
std::string str(at::ScalarType t) { return std::string("torch.") + c10::toString(t); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Failure{PyExc_TypeError, 0, std::string(name) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}

int cuda_index(const at::Tensor& t) { return t.is_cuda() ? static_cast<int>(t.get_device()) : -1; }

// Pointer of a contiguous tensor of this dtype and shape on CUDA device `index`.
void* gpu(PyObject* o, at::ScalarType dtype, std::initializer_list<int64_t> shape, int index, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dtype)
    throw Failure{PyExc_TypeError, 0, std::string(name) + " must be " + str(dtype) + ", got " + str(t.scalar_type())};
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want) refuse(std::string(name) + " must have shape " + str(want) + ", got " + str(t.sizes()));
  if (cuda_index(t) != index)
    refuse(std::string(name) + " is on " + t.device().str() + ", other tensors of the call are not");
  if (!t.is_contiguous()) throw Failure{PyExc_ValueError, 0, std::string(name) + " must be contiguous"};
  return t.data_ptr();
}

int as_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failure{nullptr, -1, ""};  // the Python error stands
  expect(v >= INT32_MIN && v <= INT32_MAX, "an integer argument is out of range");
  return static_cast<int>(v);
}

// Makes the tensors' device current for the call and names the stream: the
// handle given, or the device's current stream.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  cudaStream_t stream;
  OnDevice(int index, PyObject* given) {
    expect(index >= 0, "the tensors must be on a CUDA device");
    if (c10::cuda::current_device() != index) guard.set_index(static_cast<c10::DeviceIndex>(index));
    if (given == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    } else {
      void* p = PyLong_AsVoidPtr(given);
      if (!p && PyErr_Occurred()) throw Failure{nullptr, -1, ""};
      stream = static_cast<cudaStream_t>(p);
    }
  }
};

// A launch may wait for room in the stream: other Python threads run meanwhile.
// The error message is this thread's own.
template <typename Call>
int without_gil(Call call) {
  PyThreadState* state = PyEval_SaveThread();
  const int rc = call();
  PyEval_RestoreThread(state);
  return rc;
}

void done(int rc) {
  if (rc != DEC_OK) throw Failure{nullptr, rc, dec_last_error()};
}

struct Kv4 {
  void *kc, *kp, *vc, *vp;
  int64_t B, Hkv, S, D, NG;
  int dev;
  explicit Kv4(PyObject* const* a) {  // k_codes, k_params, v_codes, v_params
    const at::Tensor &c = tensor(a[0], "k_codes"), &p = tensor(a[1], "k_params");
    expect(c.dim() == 4 && p.dim() == 5,
           "codes must be [B, Hkv, S_max, D/2], params [B, Hkv, S_max, D/group, 2]");
    B = c.size(0), Hkv = c.size(1), S = c.size(2), D = 2 * c.size(3), NG = p.size(3);
    expect(NG >= 1 && D % NG == 0, std::to_string(NG) + " groups do not divide head_dim " + std::to_string(D));
    expect(B <= INT32_MAX && Hkv <= INT32_MAX && S <= INT32_MAX && D <= INT32_MAX, "the cache is too large");
    dev = cuda_index(c);
    kc = gpu(a[0], at::kByte, {B, Hkv, S, D / 2}, dev, "k_codes");
    kp = gpu(a[1], at::kHalf, {B, Hkv, S, NG, 2}, dev, "k_params");
    vc = gpu(a[2], at::kByte, {B, Hkv, S, D / 2}, dev, "v_codes");
    vp = gpu(a[3], at::kHalf, {B, Hkv, S, NG, 2}, dev, "v_params");
  }
  int group() const { return static_cast<int>(D / NG); }
};

// K and V rows [B, T, Hkv, D] of one type, strided alike, values contiguous.
struct Rows {
  void *k, *v;
  int bf16;
  int64_t T, sb, st, sh;
  Rows(PyObject* ko, PyObject* vo, const Kv4& c, const char* kn, const char* vn) {
    const at::Tensor &kt = tensor(ko, kn), &vt = tensor(vo, vn);
    const at::Tensor* ts[2] = {&kt, &vt};
    const char* names[2] = {kn, vn};
    for (int i = 0; i < 2; ++i) {
      const at::Tensor& t = *ts[i];
      if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
        throw Failure{PyExc_TypeError, 0,
                      std::string(names[i]) + " must be float32 or bfloat16, got " + str(t.scalar_type())};
      if (t.dim() != 4 || t.size(0) != c.B || t.size(2) != c.Hkv || t.size(3) != c.D || t.stride(3) != 1)
        refuse(std::string(names[i]) + " must be rows [" + std::to_string(c.B) + ", T, " + std::to_string(c.Hkv) + ", " +
               std::to_string(c.D) + "] with contiguous values, got " + str(t.sizes()) + " strided " + str(t.strides()));
      if (cuda_index(t) != c.dev) refuse(std::string(names[i]) + " is on " + t.device().str() + ", the cache is not");
    }
    if (kt.scalar_type() != vt.scalar_type() || kt.sizes() != vt.sizes())
      refuse(std::string(kn) + " and " + vn + " must be of one type and shape");
    // a dim of one element may carry any stride
    int64_t s[2][3];
    for (int i = 0; i < 2; ++i)
      for (int d = 0; d < 3; ++d) s[i][d] = ts[i]->size(d) > 1 ? ts[i]->stride(d) : 0;
    for (int d = 0; d < 3; ++d)
      if (s[0][d] != s[1][d]) refuse(std::string(kn) + " and " + vn + " must be strided alike");
    k = kt.data_ptr(), v = vt.data_ptr();
    bf16 = kt.scalar_type() == at::kBFloat16;
    T = kt.size(1), sb = s[0][0], st = s[0][1], sh = s[0][2];
    expect(T <= INT32_MAX, "too many tokens");
  }
};

const int32_t* ints(PyObject* o, int64_t B, int dev, const char* name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  return static_cast<const int32_t*>(gpu(o, at::kInt, {B}, dev, name));
}

// The caller's workspace, or one made on the stream that will use it (so that
// dropping it is safe); `out` gets a new reference to it.
void* workspace(PyObject* given, int Hq, int Hkv, int D, int dev, const OnDevice& on, size_t* bytes, PyObject** out) {
  if (given != Py_None) {
    const at::Tensor& t = tensor(given, "ws");
    expect(cuda_index(t) == dev && t.is_contiguous(), "ws must be contiguous memory on the tensors' device");
    *bytes = t.nbytes();
    Py_INCREF(given);
    *out = given;
    return t.data_ptr();
  }
  *bytes = dec_long_attn_workspace_size(Hq, Hkv, D);
  if (*bytes == 0) {  // sizes that the call itself refuses, with its own code
    Py_INCREF(Py_None);
    *out = Py_None;
    return nullptr;
  }
  const auto index = static_cast<c10::DeviceIndex>(dev);
  const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(on.stream, index));
  at::Tensor t = at::empty({static_cast<int64_t>(*bytes)}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, index));
  *out = THPVariable_Wrap(t);
  if (!*out) throw Failure{nullptr, -1, ""};
  return t.data_ptr();
}

// ----------------------------------------------------------------------------- calls

// k, v, pos, k_codes, k_params, v_codes, v_params, tokens, lens, from_cache, stream
PyObject* kv4_store(PyObject* const* a) {
  const Kv4 c(a + 3);
  const Rows r(a[0], a[1], c, "k", "v");
  const int T = a[7] == Py_None ? static_cast<int>(r.T) : as_int(a[7]);
  const int32_t* pos = ints(a[2], c.B, c.dev, "pos");
  const int32_t* lens = ints(a[8], c.B, c.dev, "lens", true);
  const int from_cache = PyObject_IsTrue(a[9]);
  if (from_cache < 0) throw Failure{nullptr, -1, ""};
  const OnDevice on(c.dev, a[10]);
  done(without_gil([&] {
    return dec_kv4_store(r.k, r.v, r.bf16, r.sb, r.st, r.sh, from_cache, static_cast<int>(r.T), pos, lens, T, c.kc, c.kp,
                         c.vc, c.vp, c.B, c.Hkv, c.D, c.group(), c.S, on.stream);
  }));
  Py_RETURN_NONE;
}

// k_codes, k_params, v_codes, v_params, pos, k_out, v_out, lens, stream
PyObject* kv4_load(PyObject* const* a) {
  const Kv4 c(a);
  const Rows r(a[5], a[6], c, "k_out", "v_out");
  const int32_t* pos = ints(a[4], c.B, c.dev, "pos");
  const int32_t* lens = ints(a[7], c.B, c.dev, "lens", true);
  const OnDevice on(c.dev, a[8]);
  done(without_gil([&] {
    return dec_kv4_load(c.kc, c.kp, c.vc, c.vp, pos, lens, static_cast<int>(r.T), r.k, r.v, r.bf16, r.sb, r.st, r.sh, c.B,
                        c.Hkv, c.D, c.group(), c.S, on.stream);
  }));
  Py_RETURN_NONE;
}

// q, k_codes, k_params, v_codes, v_params, pos, o, ws, stream
PyObject* kv4_decode_attn(PyObject* const* a) {
  const Kv4 c(a + 1);
  const at::Tensor& qt = tensor(a[0], "q");
  expect(qt.dim() == 3, "q must be [B, Hq, D], got " + str(qt.sizes()));
  const int64_t Hq = qt.size(1);
  expect(Hq <= INT32_MAX, "too many heads");
  const void* q = gpu(a[0], at::kFloat, {c.B, Hq, c.D}, c.dev, "q");
  const int32_t* pos = ints(a[5], c.B, c.dev, "pos");
  void* o = gpu(a[6], at::kFloat, {c.B, Hq, c.D}, c.dev, "o");
  const OnDevice on(c.dev, a[8]);
  size_t bytes;
  PyObject* held = nullptr;
  void* ws = workspace(a[7], Hq, c.Hkv, c.D, c.dev, on, &bytes, &held);
  const int rc = without_gil([&] {
    return dec_kv4_decode_attn(static_cast<const float*>(q), c.kc, c.kp, c.vc, c.vp, pos, static_cast<float*>(o), ws,
                               bytes, c.B, Hq, c.Hkv, c.D, c.group(), c.S, on.stream);
  });
  if (rc != DEC_OK) Py_DECREF(held);
  done(rc);
  return held;
}

// k_cache, pos, bounds, tokens, stream
PyObject* block_bounds(PyObject* const* a) {
  const at::Tensor& k = tensor(a[0], "k_cache");
  expect(k.dim() == 4, "k_cache must be [B, Hkv, S_max, D]");
  const int64_t B = k.size(0), Hkv = k.size(1), S = k.size(2), D = k.size(3);
  expect(B <= INT32_MAX && Hkv <= INT32_MAX && S <= INT32_MAX && D <= INT32_MAX, "the cache is too large");
  const int dev = cuda_index(k);
  const void* kp = gpu(a[0], at::kBFloat16, {B, Hkv, S, D}, dev, "k_cache");
  const int32_t* pos = ints(a[1], B, dev, "pos");
  void* bounds = gpu(a[2], at::kBFloat16, {B, Hkv, (S + 63) / 64, 2, D}, dev, "bounds");
  const int T = as_int(a[3]);
  const OnDevice on(dev, a[4]);
  done(without_gil([&] { return dec_block_bounds(kp, pos, T, bounds, B, Hkv, D, S, on.stream); }));
  Py_RETURN_NONE;
}

// q, bounds, pos, blocks, n_first, n_last, S_max (None: whole blocks), stream
PyObject* select_blocks(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &bd = tensor(a[1], "bounds"), &bl = tensor(a[3], "blocks");
  expect(q.dim() == 3 && bd.dim() == 5 && bl.dim() == 3,
         "q must be [B, Hq, D], bounds [B, Hkv, blocks, 2, D], blocks [B, Hkv, n_select]");
  const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = bd.size(1), NB = bd.size(2), n = bl.size(2);
  expect(B <= INT32_MAX && Hq <= INT32_MAX && D <= INT32_MAX && Hkv <= INT32_MAX && NB <= INT32_MAX / 64 &&
             n <= INT32_MAX,
         "the sizes are too large");
  const int dev = cuda_index(q);
  const void* qp = gpu(a[0], at::kFloat, {B, Hq, D}, dev, "q");
  const void* bounds = gpu(a[1], at::kBFloat16, {B, Hkv, NB, 2, D}, dev, "bounds");
  const int32_t* pos = ints(a[2], B, dev, "pos");
  void* blocks = gpu(a[3], at::kInt, {B, Hkv, n}, dev, "blocks");
  const int first = as_int(a[4]), last = as_int(a[5]);
  const int S = a[6] == Py_None ? static_cast<int>(NB * 64) : as_int(a[6]);
  expect(S >= 1 && (S - 1) / 64 + 1 == NB, std::to_string(NB) + " blocks of bounds do not match S_max = " +
                                               std::to_string(S) + " slots");
  const OnDevice on(dev, a[7]);
  done(without_gil([&] {
    return dec_select_blocks(static_cast<const float*>(qp), bounds, pos, static_cast<int32_t*>(blocks), n, first, last, B,
                             Hq, Hkv, D, S, on.stream);
  }));
  Py_RETURN_NONE;
}

// q, k_cache, v_cache, pos, blocks, o, ws, stream
PyObject* block_decode_attn(PyObject* const* a) {
  const at::Tensor &qt = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &bl = tensor(a[4], "blocks");
  expect(qt.dim() == 3 && k.dim() == 4 && bl.dim() == 3,
         "q must be [B, Hq, D], the caches [B, Hkv, S_max, D], blocks [B, Hkv, n_select]");
  const int64_t B = k.size(0), Hkv = k.size(1), S = k.size(2), D = k.size(3), Hq = qt.size(1), n = bl.size(2);
  expect(B <= INT32_MAX && Hq <= INT32_MAX && Hkv <= INT32_MAX && S <= INT32_MAX && D <= INT32_MAX && n <= INT32_MAX,
         "the sizes are too large");
  const int dev = cuda_index(k);
  const void* q = gpu(a[0], at::kFloat, {B, Hq, D}, dev, "q");
  const void* kp = gpu(a[1], at::kBFloat16, {B, Hkv, S, D}, dev, "k_cache");
  const void* vp = gpu(a[2], at::kBFloat16, {B, Hkv, S, D}, dev, "v_cache");
  const int32_t* pos = ints(a[3], B, dev, "pos");
  const void* blocks = gpu(a[4], at::kInt, {B, Hkv, n}, dev, "blocks");
  void* o = gpu(a[5], at::kFloat, {B, Hq, D}, dev, "o");
  const OnDevice on(dev, a[7]);
  size_t bytes;
  PyObject* held = nullptr;
  void* ws = workspace(a[6], Hq, Hkv, D, dev, on, &bytes, &held);
  const int rc = without_gil([&] {
    return dec_block_decode_attn(static_cast<const float*>(q), kp, vp, pos, static_cast<const int32_t*>(blocks), n,
                                 static_cast<float*>(o), ws, bytes, B, Hq, Hkv, D, S, on.stream);
  });
  if (rc != DEC_OK) Py_DECREF(held);
  done(rc);
  return held;
}

// One Python entry: N positional arguments, no C++ exception leaves it.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Failure& f) {
    if (f.code < 0) return nullptr;
    if (f.type) {
      PyErr_SetString(f.type, f.text.c_str());
      return nullptr;
    }
    PyObject* e = g_dec_error ? PyObject_CallFunction(g_dec_error, "is", f.code, f.text.c_str()) : nullptr;
    if (e) {
      PyErr_SetObject(g_dec_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_SetString(PyExc_RuntimeError, f.text.c_str());
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_dec_error);
  g_dec_error = cls;
  Py_RETURN_NONE;
}

#define DEC_ENTRY(name, n) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name, n>)), METH_FASTCALL, nullptr }

PyMethodDef kMethods[] = {DEC_ENTRY(kv4_store, 11),
                          DEC_ENTRY(kv4_load, 9),
                          DEC_ENTRY(kv4_decode_attn, 9),
                          DEC_ENTRY(block_bounds, 5),
                          DEC_ENTRY(select_blocks, 8),
                          DEC_ENTRY(block_decode_attn, 8),
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {
    PyModuleDef_HEAD_INIT, "_binding", "Native marshalling of libdec's long-cache calls.", -1, kMethods, nullptr, nullptr,
    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
