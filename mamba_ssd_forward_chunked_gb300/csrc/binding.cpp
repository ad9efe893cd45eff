// The layer operators on torch tensors (module _layer_binding): checks every
// tensor, allocates the outputs that are not given, fills the argument struct
// and calls the C entry point of include/ssd.h on the current stream.
//
// In C++ because these are the calls a decoding loop makes for every layer and
// token: a dozen tensors' checks cost about 6 us a call in Python, more than
// most of the kernels, and under 1 us here.  Signatures, defaults and
// documentation are in layer.py; arguments come by position, None for what is
// not given.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>
#include <vector>

#include "ssd.h"

namespace {

PyObject* g_error = nullptr;  // the package's SSDError

struct Refused {
  int code;
  std::string why;
};
struct PythonError {};  // the interpreter holds it already

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{1, std::string(name) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}

// The tensor the other arguments go by.
struct First {
  const at::Tensor& t;
  at::ScalarType type;
  int dtype, dev;
};
First first(PyObject* o, const char* name, int64_t dims) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != dims)
    throw Refused{1, std::string(name) + " must be a " + std::to_string(dims) + "-D tensor"};
  const at::Tensor& t = THPVariable_Unpack(o);
  const at::ScalarType type = t.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16)
    throw Refused{2, std::string(name) + " has dtype " + c10::toString(type) + ", expected float32 or bfloat16"};
  if (!t.is_cuda()) throw Refused{1, std::string(name) + " must be a CUDA tensor (got " + t.device().str() + ")"};
  return {t, type, type == at::kBFloat16 ? SSD_BF16 : SSD_F32, t.get_device()};
}

const at::Tensor& checked(PyObject* o, const char* name, int dev, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.get_device() != dev)
    throw Refused{1, std::string(name) + " is on " + t.device().str() + ", the other arguments on cuda:" + std::to_string(dev)};
  if (t.scalar_type() != type)
    throw Refused{1, std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(type)};
  if (t.sizes() != shape)
    throw Refused{1, std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape)};
  return t;
}

// The address of a contiguous tensor of this type and shape (null for None).
template <typename P = const void>
P* dense(PyObject* o, const char* name, int dev, at::ScalarType type, at::IntArrayRef shape) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = checked(o, name, dev, type, shape);
  if (!t.is_contiguous()) throw Refused{1, std::string(name) + " must be contiguous"};
  return static_cast<P*>(t.data_ptr());
}

// The address of a tensor whose last dimension is contiguous; its other strides stay in `t`.
const void* rows(PyObject* o, const char* name, int dev, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor& t = checked(o, name, dev, type, shape);
  if (shape.back() > 1 && t.strides().back() != 1)
    throw Refused{1, std::string(name) + " must be contiguous in its last dimension"};
  return t.data_ptr();
}
// The address of a tensor [batch][seqlen][...] whose last two dimensions are contiguous.
const void* inner(PyObject* o, const char* name, int dev, at::ScalarType type, at::IntArrayRef shape) {
  const void* at = rows(o, name, dev, type, shape);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (shape[2] > 1 && t.stride(2) != shape[3])
    throw Refused{1, std::string(name) + " must be contiguous in its last two dimensions"};
  return at;
}
int64_t stride(PyObject* o, int d) { return THPVariable_Unpack(o).stride(d); }

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::empty(shape, like.options().dtype(type));
}

int64_t whole(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{1, std::string(name) + " must be a whole number"};
  }
  return v;
}

float real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{1, std::string(name) + " must be a number"};
  }
  return static_cast<float>(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};  // as of a tensor of several values
  return v == 1;
}

int small(int64_t v, const char* name) {
  if (v > INT32_MAX || v < INT32_MIN) throw Refused{2, std::string(name) + " is " + std::to_string(v)};
  return static_cast<int>(v);
}

// The items of a list or tuple (or one tensor by itself).
struct Items {
  PyObject* seq = nullptr;
  std::vector<PyObject*> v;
  Items(PyObject* o, const char* name) {
    if (THPVariable_Check(o)) {
      v.push_back(o);
      return;
    }
    seq = PySequence_Fast(o, "");
    if (!seq) {
      PyErr_Clear();
      throw Refused{1, std::string(name) + " must be a sequence"};
    }
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(seq); ++i) v.push_back(PySequence_Fast_GET_ITEM(seq, i));
  }
  ~Items() { Py_XDECREF(seq); }
};

// The tensors' device is the current one while this lives: workspaces are sized for it, and the call runs on it.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  explicit On(int dev) {
    if (c10::cuda::current_device() != dev) guard.set_index(static_cast<c10::DeviceIndex>(dev));
  }
};

template <typename Args>
void call(ssd_status (*fn)(const Args*, ssd_stream_t), const char* name, Args& a, int dev) {
  a.size = sizeof(Args);
  const ssd_status st = fn(&a, c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
  if (st != SSD_OK) throw Refused{st, name};
}

PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw PythonError{};
  return o;
}
// A new tuple of tensors.
PyObject* wrap_all(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw PythonError{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// u, weight, bias, activation, split, ring, positions, lengths, slots, new_ring, out
PyObject* conv_fwd(PyObject* const* p) {
  const First u = first(p[0], "u", 3);
  const On device(u.dev);
  const int64_t B = u.t.size(0), L = u.t.size(1), C = u.t.size(2);
  ssd_conv_args a{};
  a.batch = B, a.seqlen = L, a.channels = small(C, "channels"), a.dtype = u.dtype;
  if (p[3] == Py_None) {
    a.activation = SSD_ACT_NONE;
  } else if (PyUnicode_Check(p[3]) && PyUnicode_CompareWithASCIIString(p[3], "silu") == 0) {
    a.activation = SSD_ACT_SILU;
  } else {
    throw Refused{2, "activation must be 'silu' or None"};
  }
  std::vector<int64_t> parts;
  if (p[4] == Py_None) {
    parts.push_back(C);
  } else {
    Items split(p[4], "split");
    int64_t sum = 0;
    for (PyObject* o : split.v) {
      parts.push_back(whole(o, "split"));
      if (parts.back() < 1 || parts.back() > C) sum = -(int64_t(1) << 40);
      sum += parts.back();
    }
    if (parts.empty() || parts.size() > 3 || sum != C)
      throw Refused{1, "split " + text(parts) + " does not divide " + std::to_string(C) + " channels in one to three parts"};
  }
  a.nout = static_cast<int>(parts.size());
  a.u = rows(p[0], "u", u.dev, u.type, {B, L, C});
  a.u_batch = u.t.stride(0), a.u_token = u.t.stride(1);
  const int64_t W = THPVariable_Check(p[1]) && THPVariable_Unpack(p[1]).dim() == 2 ? THPVariable_Unpack(p[1]).size(1) : 0;
  a.width = small(W, "width");
  a.weight = dense<const float>(p[1], "weight", u.dev, at::kFloat, {C, W});
  a.bias = dense<const float>(p[2], "bias", u.dev, at::kFloat, {C});
  if (p[5] == Py_None) {
    if (p[8] != Py_None || p[9] != Py_None) throw Refused{1, "new_ring and slots belong to a ring"};
  } else {
    const at::Tensor& ring = tensor(p[5], "ring");
    a.nslots = ring.dim() == 3 ? ring.size(0) : 0;
    a.ring = dense<const void>(p[5], "ring", u.dev, u.type, {a.nslots, W, C});
    a.new_ring = dense<void>(p[9], "new_ring", u.dev, u.type, {a.nslots, W, C});
  }
  a.positions = dense<const int32_t>(p[6], "positions", u.dev, at::kInt, {B});
  a.lengths = dense<const int32_t>(p[7], "lengths", u.dev, at::kInt, {B});
  a.slots = dense<const int32_t>(p[8], "slots", u.dev, at::kInt, {B});
  at::Tensor out[3];
  if (p[10] == Py_None) {
    for (int i = 0; i < a.nout; ++i) out[i] = empty({B, L, parts[i]}, u.type, u.t);
  } else {
    Items given(p[10], "out");
    if (given.v.size() != parts.size())
      throw Refused{1, std::to_string(given.v.size()) + " outputs for " + std::to_string(parts.size()) + " parts"};
    for (int i = 0; i < a.nout; ++i) {
      dense<void>(given.v[i], "out", u.dev, u.type, {B, L, parts[i]});
      out[i] = tensor(given.v[i], "out");
    }
  }
  for (int i = 0; i < a.nout; ++i) a.out_channels[i] = static_cast<int32_t>(parts[i]), a.out[i] = out[i].data_ptr();
  call(ssd_conv_fwd, "ssd_conv_fwd", a, u.dev);
  if (p[4] == Py_None) return wrap(out[0]);
  return a.nout == 1 ? wrap_all({out[0]}) : a.nout == 2 ? wrap_all({out[0], out[1]}) : wrap_all({out[0], out[1], out[2]});
}

// u, delta, A, Bm, Cm, D, z, delta_bias, delta_softplus, init_state, lengths, y, final_state, workspace, want_final_state
PyObject* selective_scan(PyObject* const* p) {
  const First u = first(p[0], "u", 3);
  const On device(u.dev);
  const int64_t B = u.t.size(0), L = u.t.size(1), C = u.t.size(2);
  if (!THPVariable_Check(p[3]) || THPVariable_Unpack(p[3]).dim() != 4) throw Refused{1, "Bm must be a 4-D tensor"};
  const int64_t G = THPVariable_Unpack(p[3]).size(2), N = THPVariable_Unpack(p[3]).size(3);
  ssd_selective_scan_args a{};
  a.batch = B, a.seqlen = L, a.channels = small(C, "channels"), a.dstate = small(N, "dstate");
  a.ngroups = small(G, "ngroups"), a.dtype = u.dtype, a.softplus = truth(p[8]);
  a.u = rows(p[0], "u", u.dev, u.type, {B, L, C});
  a.u_batch = u.t.stride(0), a.u_token = u.t.stride(1);
  a.delta = rows(p[1], "delta", u.dev, u.type, {B, L, C});
  a.delta_batch = stride(p[1], 0), a.delta_token = stride(p[1], 1);
  if (p[6] != Py_None) {
    a.z = rows(p[6], "z", u.dev, u.type, {B, L, C});
    a.z_batch = stride(p[6], 0), a.z_token = stride(p[6], 1);
  }
  a.Bm = rows(p[3], "Bm", u.dev, u.type, {B, L, G, N});
  a.B_batch = stride(p[3], 0), a.B_token = stride(p[3], 1);
  a.Cm = rows(p[4], "Cm", u.dev, u.type, {B, L, G, N});
  a.C_batch = stride(p[4], 0), a.C_token = stride(p[4], 1);
  if (G > 1 && (stride(p[3], 2) != N || stride(p[4], 2) != N))
    throw Refused{1, "Bm and Cm must be contiguous over their groups"};
  if (p[2] == Py_None) throw Refused{1, "A must be a torch.Tensor"};
  a.A = dense<const float>(p[2], "A", u.dev, at::kFloat, {C, N});
  a.D = dense<const float>(p[5], "D", u.dev, at::kFloat, {C});
  a.delta_bias = dense<const float>(p[7], "delta_bias", u.dev, at::kFloat, {C});
  a.init_state = dense<const float>(p[9], "init_state", u.dev, at::kFloat, {B, C, N});
  a.lengths = dense<const int32_t>(p[10], "lengths", u.dev, at::kInt, {B});
  a.y = dense<void>(p[11], "y", u.dev, u.type, {B, L, C});
  a.final_state = dense<float>(p[12], "final_state", u.dev, at::kFloat, {B, C, N});
  const at::Tensor y = a.y || p[11] != Py_None ? tensor(p[11], "y") : empty({B, L, C}, u.type, u.t);
  a.y = y.data_ptr();
  at::Tensor final_state;
  if (p[12] != Py_None) {
    final_state = tensor(p[12], "final_state");
  } else if (truth(p[14])) {
    final_state = empty({B, C, N}, at::kFloat, u.t);
    a.final_state = static_cast<float*>(final_state.data_ptr());
  }
  a.size = sizeof(a);
  at::Tensor space;
  if (p[13] != Py_None) {
    const int64_t bytes = tensor(p[13], "workspace").numel();
    a.workspace = dense<void>(p[13], "workspace", u.dev, at::kByte, {bytes});
    a.workspace_bytes = static_cast<size_t>(bytes);
  } else if (const size_t need = ssd_selective_scan_workspace_size(&a)) {
    space = empty({static_cast<int64_t>(need)}, at::kByte, u.t);
    a.workspace = space.data_ptr(), a.workspace_bytes = need;
  }
  call(ssd_selective_scan, "ssd_selective_scan", a, u.dev);
  if (final_state.defined()) return wrap_all({y, final_state});
  PyObject* r = PyTuple_New(2);
  if (!r) throw PythonError{};
  PyTuple_SET_ITEM(r, 1, Py_NewRef(Py_None));
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(y));
  return r;
}

// u, dt, A, D, weight, bias, state, ring, positions, ngroups, z, dt_bias, dt_softplus, slots, new_state, y
PyObject* step(PyObject* const* p) {
  const First u = first(p[0], "u", 2);
  const On device(u.dev);
  if (!THPVariable_Check(p[6]) || THPVariable_Unpack(p[6]).dim() != 4) throw Refused{1, "state must be a 4-D tensor"};
  const at::Tensor& state = THPVariable_Unpack(p[6]);
  const int64_t B = u.t.size(0), C = u.t.size(1), S = state.size(0), H = state.size(1), P = state.size(2), N = state.size(3);
  const int64_t G = whole(p[9], "ngroups");
  if (G < 1 || G > C || C != H * P + 2 * G * N)
    throw Refused{1, "u has " + std::to_string(C) + " channels, which are not nheads*headdim + 2*ngroups*dstate"};
  ssd_step_args a{};
  a.batch = B, a.nslots = S, a.nheads = small(H, "nheads"), a.headdim = small(P, "headdim");
  a.ngroups = small(G, "ngroups"), a.dstate = small(N, "dstate"), a.dtype = u.dtype;
  const int64_t W = THPVariable_Check(p[4]) && THPVariable_Unpack(p[4]).dim() == 2 ? THPVariable_Unpack(p[4]).size(1) : 0;
  a.width = small(W, "width");
  a.softplus = truth(p[12]);
  a.u = rows(p[0], "u", u.dev, u.type, {B, C});
  a.u_batch = u.t.stride(0);
  if (p[10] != Py_None) {
    a.z = rows(p[10], "z", u.dev, u.type, {B, H * P});
    a.z_batch = stride(p[10], 0);
  }
  const bool dt32 = THPVariable_Check(p[1]) && THPVariable_Unpack(p[1]).scalar_type() == at::kFloat;
  a.dt_dtype = dt32 ? static_cast<int>(SSD_F32) : u.dtype;
  a.dt = rows(p[1], "dt", u.dev, dt32 ? at::kFloat : u.type, {B, H});
  a.dt_batch = stride(p[1], 0);
  for (int i : {2, 3, 4, 7, 8})
    if (p[i] == Py_None) throw Refused{1, "A, D, weight, ring and positions must be tensors"};
  a.A = dense<const float>(p[2], "A", u.dev, at::kFloat, {H});
  a.D = dense<const float>(p[3], "D", u.dev, at::kFloat, {H});
  a.weight = dense<const float>(p[4], "weight", u.dev, at::kFloat, {C, W});
  a.bias = dense<const float>(p[5], "bias", u.dev, at::kFloat, {C});
  a.state = dense<const float>(p[6], "state", u.dev, at::kFloat, {S, H, P, N});
  a.ring = dense<void>(p[7], "ring", u.dev, u.type, {S, W, C});
  a.positions = dense<const int32_t>(p[8], "positions", u.dev, at::kInt, {B});
  a.dt_bias = dense<const float>(p[11], "dt_bias", u.dev, at::kFloat, {H});
  a.slots = dense<const int32_t>(p[13], "slots", u.dev, at::kInt, {B});
  a.new_state = dense<float>(p[14], "new_state", u.dev, at::kFloat, {S, H, P, N});
  dense<void>(p[15], "y", u.dev, u.type, {B, H, P});
  const at::Tensor y = p[15] != Py_None ? tensor(p[15], "y") : empty({B, H, P}, u.type, u.t);
  a.y = y.data_ptr();
  call(ssd_step, "ssd_step", a, u.dev);
  return wrap(y);
}

// x, packed, scales, group, add, y, workspace
PyObject* w4_matvec(PyObject* const* p) {
  const First x = first(p[0], "x", 2);
  const On device(x.dev);
  const int64_t M = x.t.size(0), K = x.t.size(1), group = whole(p[3], "group");
  if (!THPVariable_Check(p[2]) || THPVariable_Unpack(p[2]).dim() != 2) throw Refused{1, "scales must be a 2-D tensor"};
  if (group != 32 && group != 64 && group != 128)
    throw Refused{2, "group " + std::to_string(group) + ", expected 32, 64 or 128"};
  const int64_t n = THPVariable_Unpack(p[2]).size(0);
  ssd_w4_matvec_args a{};
  a.tokens = M, a.n = small(n, "n"), a.k = small(K, "k"), a.group = static_cast<int32_t>(group), a.dtype = x.dtype;
  a.x = rows(p[0], "x", x.dev, x.type, {M, K});
  a.x_token = x.t.stride(0);
  if (p[1] == Py_None) throw Refused{1, "packed must be a torch.Tensor"};
  a.packed = dense(p[1], "packed", x.dev, at::kInt, {(n + 15) / 16, (K + 63) / 64, 32, 4});
  a.scales = dense<const float>(p[2], "scales", x.dev, at::kFloat, {n, (K + group - 1) / group});
  if (p[4] != Py_None) {
    a.add = rows(p[4], "add", x.dev, x.type, {M, n});
    a.add_token = stride(p[4], 0);
  }
  dense<void>(p[5], "y", x.dev, x.type, {M, n});
  const at::Tensor y = p[5] != Py_None ? tensor(p[5], "y") : empty({M, n}, x.type, x.t);
  a.y = y.data_ptr();
  a.size = sizeof(a);
  at::Tensor space;
  if (p[6] != Py_None) {
    const int64_t bytes = tensor(p[6], "workspace").numel();
    a.workspace = dense<void>(p[6], "workspace", x.dev, at::kByte, {bytes});
    a.workspace_bytes = static_cast<size_t>(bytes);
  } else if (const size_t need = ssd_w4_matvec_workspace_size(&a)) {
    space = empty({static_cast<int64_t>(need)}, at::kByte, x.t);
    a.workspace = space.data_ptr(), a.workspace_bytes = need;
  }
  call(ssd_w4_matvec, "ssd_w4_matvec", a, x.dev);
  return wrap(y);
}

// logits, scores, k, finished, eos, workspace
PyObject* beam_select(PyObject* const* p) {
  const First x = first(p[0], "logits", 3);
  const On device(x.dev);
  const int64_t B = x.t.size(0), W = x.t.size(1), V = x.t.size(2), k = whole(p[2], "k");
  if (k < 1 || k > 64) throw Refused{k < 1 ? 1 : 2, "k is " + std::to_string(k) + ", expected 1 to 64"};
  ssd_beam_select_args a{};
  a.batch = B, a.beams = small(W, "beams"), a.vocab = small(V, "vocab"), a.k = static_cast<int32_t>(k);
  a.dtype = x.dtype, a.eos = small(whole(p[4], "eos"), "eos");
  a.logits = rows(p[0], "logits", x.dev, x.type, {B, W, V});
  a.logits_batch = x.t.stride(0), a.logits_beam = x.t.stride(1);
  if (p[1] == Py_None) throw Refused{1, "scores must be a torch.Tensor"};
  a.scores = dense<const float>(p[1], "scores", x.dev, at::kFloat, {B, W});
  a.finished = dense<const uint8_t>(p[3], "finished", x.dev, at::kBool, {B, W});
  a.size = sizeof(a);
  at::Tensor space;
  if (p[5] != Py_None) {
    const int64_t bytes = tensor(p[5], "workspace").numel();
    a.workspace = dense<void>(p[5], "workspace", x.dev, at::kByte, {bytes});
    a.workspace_bytes = static_cast<size_t>(bytes);
  } else {
    a.workspace_bytes = ssd_beam_select_workspace_size(&a);
    space = empty({static_cast<int64_t>(a.workspace_bytes)}, at::kByte, x.t);
    a.workspace = space.data_ptr();
  }
  const at::Tensor best = empty({B, k}, at::kFloat, x.t), parents = empty({B, k}, at::kInt, x.t),
                   tokens = empty({B, k}, at::kInt, x.t);
  a.out_scores = static_cast<float*>(best.data_ptr());
  a.parents = static_cast<int32_t*>(parents.data_ptr()), a.tokens = static_cast<int32_t*>(tokens.data_ptr());
  call(ssd_beam_select, "ssd_beam_select", a, x.dev);
  return wrap_all({best, parents, tokens});
}

// states, parents, out (or None: in place)
PyObject* beam_reorder(PyObject* const* p) {
  if (!THPVariable_Check(p[1]) || THPVariable_Unpack(p[1]).dim() != 2) throw Refused{1, "parents must be a 2-D tensor"};
  const at::Tensor& parents = THPVariable_Unpack(p[1]);
  if (!parents.is_cuda()) throw Refused{1, "parents must be a CUDA tensor (got " + parents.device().str() + ")"};
  const int dev = parents.get_device();
  const On device(dev);
  const int64_t B = parents.size(0), k = parents.size(1);
  const int32_t* pp = dense<const int32_t>(p[1], "parents", dev, at::kInt, {B, k});
  Items states(p[0], "states");
  Items out(p[2] == Py_None ? p[0] : p[2], "out");
  if (out.v.size() != states.v.size())
    throw Refused{1, std::to_string(out.v.size()) + " outputs for " + std::to_string(states.v.size()) + " states"};
  const size_t count = states.v.size();
  int64_t beams = 0;
  std::vector<ssd_beam_reorder_args> calls((count + SSD_REORDER_MAX - 1) / SSD_REORDER_MAX);
  for (size_t i = 0; i < count; ++i) {
    const at::Tensor& t = tensor(states.v[i], "state");
    if (t.dim() < 1 || (B ? t.size(0) % B != 0 : t.size(0) != 0))
      throw Refused{1, "a state must have a multiple of " + std::to_string(B) + " rows"};
    const int64_t w = B ? t.size(0) / B : k;
    if (i && w != beams) throw Refused{1, "the states must have the same number of rows"};
    beams = w;
    ssd_beam_reorder_args& a = calls[i / SSD_REORDER_MAX];
    const int j = a.count++;
    a.src[j] = dense(states.v[i], "state", dev, t.scalar_type(), t.sizes());
    std::vector<int64_t> shape = t.sizes().vec();
    shape[0] = B * k;
    a.dst[j] = dense<void>(out.v[i], "out", dev, t.scalar_type(), shape);
    a.row_bytes[j] = t.size(0) ? t.numel() / t.size(0) * static_cast<int64_t>(t.element_size()) : 0;
  }
  for (ssd_beam_reorder_args& a : calls) {
    a.batch = B, a.beams = small(beams, "beams"), a.k = small(k, "k"), a.parents = pp;
    call(ssd_beam_reorder, "ssd_beam_reorder", a, dev);
  }
  PyObject* r = PyList_New(static_cast<Py_ssize_t>(count));
  if (!r) throw PythonError{};
  for (size_t i = 0; i < count; ++i) PyList_SET_ITEM(r, static_cast<Py_ssize_t>(i), Py_NewRef(out.v[i]));
  return r;
}

// x, dt, A, Bm, Cm, beta, scale, dt_bias, dt_softplus, beta_sigmoid, norm_eps, init_state, slots, positions, lengths, y,
// final_state, workspace, want_final_state
PyObject* delta_fwd(PyObject* const* p) {
  const First x = first(p[0], "x", 4);
  const On device(x.dev);
  const int64_t B = x.t.size(0), L = x.t.size(1), H = x.t.size(2), P = x.t.size(3);
  if (!THPVariable_Check(p[3]) || THPVariable_Unpack(p[3]).dim() != 4) throw Refused{1, "Bm must be a 4-D tensor"};
  const int64_t G = THPVariable_Unpack(p[3]).size(2), N = THPVariable_Unpack(p[3]).size(3);
  ssd_delta_args a{};
  a.batch = B, a.seqlen = L, a.nheads = small(H, "nheads"), a.headdim = small(P, "headdim");
  a.ngroups = small(G, "ngroups"), a.dstate = small(N, "dstate"), a.dtype = x.dtype;
  a.scale = p[6] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(N))) : real(p[6], "scale");
  a.norm_eps = p[10] == Py_None ? -1.f : real(p[10], "norm_eps");
  if (p[10] != Py_None && !(a.norm_eps >= 0.f)) throw Refused{1, "norm_eps must not be negative"};
  a.dt_softplus = truth(p[8]), a.beta_sigmoid = truth(p[9]);
  a.x = inner(p[0], "x", x.dev, x.type, {B, L, H, P});
  a.x_batch = x.t.stride(0), a.x_token = x.t.stride(1);
  a.Bm = inner(p[3], "Bm", x.dev, x.type, {B, L, G, N});
  a.B_batch = stride(p[3], 0), a.B_token = stride(p[3], 1);
  a.Cm = inner(p[4], "Cm", x.dev, x.type, {B, L, G, N});
  a.C_batch = stride(p[4], 0), a.C_token = stride(p[4], 1);
  const bool gates32 = THPVariable_Check(p[1]) && THPVariable_Unpack(p[1]).scalar_type() == at::kFloat;
  a.gate_dtype = gates32 ? static_cast<int>(SSD_F32) : x.dtype;
  const at::ScalarType gates = gates32 ? at::kFloat : x.type;
  a.dt = rows(p[1], "dt", x.dev, gates, {B, L, H});
  a.dt_batch = stride(p[1], 0), a.dt_token = stride(p[1], 1);
  a.beta = rows(p[5], "beta", x.dev, gates, {B, L, H});
  a.beta_batch = stride(p[5], 0), a.beta_token = stride(p[5], 1);
  if (p[2] == Py_None) throw Refused{1, "A must be a torch.Tensor"};
  a.A = dense<const float>(p[2], "A", x.dev, at::kFloat, {H});
  a.dt_bias = dense<const float>(p[7], "dt_bias", x.dev, at::kFloat, {H});
  const bool want = truth(p[18]);
  a.nslots = B;
  for (int i : {11, 16})
    if (p[i] != Py_None) a.nslots = tensor(p[i], i == 11 ? "init_state" : "final_state").dim() == 4 ? THPVariable_Unpack(p[i]).size(0) : 0;
  a.init_state = dense<const float>(p[11], "init_state", x.dev, at::kFloat, {a.nslots, H, P, N});
  a.final_state = dense<float>(p[16], "final_state", x.dev, at::kFloat, {a.nslots, H, P, N});
  a.slots = dense<const int32_t>(p[12], "slots", x.dev, at::kInt, {B});
  a.positions = dense<const int32_t>(p[13], "positions", x.dev, at::kInt, {B});
  a.lengths = dense<const int32_t>(p[14], "lengths", x.dev, at::kInt, {B});
  if (p[12] != Py_None && p[11] == Py_None && p[16] == Py_None) throw Refused{1, "slots belong to states"};
  dense<void>(p[15], "y", x.dev, x.type, {B, L, H, P});
  const at::Tensor y = p[15] != Py_None ? tensor(p[15], "y") : empty({B, L, H, P}, x.type, x.t);
  a.y = y.data_ptr();
  at::Tensor final_state;
  if (p[16] != Py_None) {
    final_state = tensor(p[16], "final_state");
  } else if (want) {
    if (p[12] != Py_None) throw Refused{1, "with slots, final_state must be given"};
    final_state = empty({a.nslots, H, P, N}, at::kFloat, x.t);
    a.final_state = static_cast<float*>(final_state.data_ptr());
  }
  a.size = sizeof(a);
  at::Tensor space;
  if (p[17] != Py_None) {
    const int64_t bytes = tensor(p[17], "workspace").numel();
    a.workspace = dense<void>(p[17], "workspace", x.dev, at::kByte, {bytes});
    a.workspace_bytes = static_cast<size_t>(bytes);
  } else if (const size_t need = ssd_delta_workspace_size(&a)) {
    space = empty({static_cast<int64_t>(need)}, at::kByte, x.t);
    a.workspace = space.data_ptr(), a.workspace_bytes = need;
  }
  call(ssd_delta_fwd, "ssd_delta_fwd", a, x.dev);
  if (final_state.defined()) return wrap_all({y, final_state});
  PyObject* r = PyTuple_New(2);
  if (!r) throw PythonError{};
  PyTuple_SET_ITEM(r, 1, Py_NewRef(Py_None));
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(y));
  return r;
}

// logits, draft, uniforms, draft_logits, scale, lengths, workspace
PyObject* draft_verify(PyObject* const* p) {
  const First x = first(p[0], "logits", 3);
  const On device(x.dev);
  const int64_t B = x.t.size(0), T = x.t.size(1) - 1, V = x.t.size(2);
  if (T < 0) throw Refused{1, "logits must have a row for every draft and one more"};
  ssd_draft_verify_args a{};
  a.batch = B, a.drafts = small(T, "drafts"), a.vocab = small(V, "vocab"), a.dtype = x.dtype;
  a.logits = rows(p[0], "logits", x.dev, x.type, {B, T + 1, V});
  a.logits_batch = x.t.stride(0), a.logits_row = x.t.stride(1);
  for (int i : {1, 2})
    if (p[i] == Py_None) throw Refused{1, "draft and uniforms must be tensors"};
  a.draft = dense<const int32_t>(p[1], "draft", x.dev, at::kInt, {B, T});
  a.uniforms = dense<const float>(p[2], "uniforms", x.dev, at::kFloat, {B, T + 1});
  if (p[3] != Py_None && T > 0) {
    a.draft_logits = rows(p[3], "draft_logits", x.dev, x.type, {B, T, V});
    a.draft_logits_batch = stride(p[3], 0), a.draft_logits_row = stride(p[3], 1);
  }
  a.scale = dense<const float>(p[4], "scale", x.dev, at::kFloat, {B});
  a.lengths = dense<const int32_t>(p[5], "lengths", x.dev, at::kInt, {B});
  a.size = sizeof(a);
  at::Tensor space;
  if (p[6] != Py_None) {
    const int64_t bytes = tensor(p[6], "workspace").numel();
    a.workspace = dense<void>(p[6], "workspace", x.dev, at::kByte, {bytes});
    a.workspace_bytes = static_cast<size_t>(bytes);
  } else {
    a.workspace_bytes = ssd_draft_verify_workspace_size(&a);
    space = empty({static_cast<int64_t>(a.workspace_bytes)}, at::kByte, x.t);
    a.workspace = space.data_ptr();
  }
  const at::Tensor tokens = empty({B, T + 1}, at::kInt, x.t), accepted = empty({B}, at::kInt, x.t),
                   logprobs = empty({B, T + 1}, at::kFloat, x.t);
  a.tokens = static_cast<int32_t*>(tokens.data_ptr()), a.accepted = static_cast<int32_t*>(accepted.data_ptr());
  a.logprobs = static_cast<float*>(logprobs.data_ptr());
  call(ssd_draft_verify, "ssd_draft_verify", a, x.dev);
  return wrap_all({tokens, accepted, logprobs});
}

// batch, seqlen, channels, dstate, ngroups
PyObject* scan_workspace(PyObject* const* p) {
  ssd_selective_scan_args a{};
  a.size = sizeof(a);
  a.batch = whole(p[0], "batch"), a.seqlen = whole(p[1], "seqlen"), a.channels = small(whole(p[2], "channels"), "channels");
  a.dstate = small(whole(p[3], "dstate"), "dstate"), a.ngroups = small(whole(p[4], "ngroups"), "ngroups");
  return PyLong_FromSize_t(ssd_selective_scan_workspace_size(&a));
}

// batch, beams, vocab, k
PyObject* select_workspace(PyObject* const* p) {
  ssd_beam_select_args a{};
  a.size = sizeof(a);
  a.batch = whole(p[0], "batch"), a.beams = small(whole(p[1], "beams"), "beams");
  a.vocab = small(whole(p[2], "vocab"), "vocab"), a.k = small(whole(p[3], "k"), "k");
  return PyLong_FromSize_t(ssd_beam_select_workspace_size(&a));
}

// batch, seqlen, nheads, headdim, ngroups, dstate, bf16
PyObject* delta_workspace(PyObject* const* p) {
  ssd_delta_args a{};
  a.size = sizeof(a);
  a.batch = whole(p[0], "batch"), a.seqlen = whole(p[1], "seqlen"), a.nslots = a.batch;
  a.nheads = small(whole(p[2], "nheads"), "nheads"), a.headdim = small(whole(p[3], "headdim"), "headdim");
  a.ngroups = small(whole(p[4], "ngroups"), "ngroups"), a.dstate = small(whole(p[5], "dstate"), "dstate");
  a.dtype = a.gate_dtype = truth(p[6]) ? SSD_BF16 : SSD_F32;
  return PyLong_FromSize_t(ssd_delta_workspace_size(&a));
}

// batch, drafts, vocab, bf16, draft_logits
PyObject* verify_workspace(PyObject* const* p) {
  ssd_draft_verify_args a{};
  a.size = sizeof(a);
  a.batch = whole(p[0], "batch"), a.drafts = small(whole(p[1], "drafts"), "drafts");
  a.vocab = small(whole(p[2], "vocab"), "vocab"), a.dtype = truth(p[3]) ? SSD_BF16 : SSD_F32;
  a.draft_logits = truth(p[4]) && a.drafts > 0 ? &a : nullptr;  // whether there are any is all that is read
  return PyLong_FromSize_t(ssd_draft_verify_workspace_size(&a));
}

// No C++ exception leaves the module.
template <PyObject* (*fn)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return fn(args);
  } catch (const Refused& e) {
    PyObject* v = Py_BuildValue("(is)", e.code, e.why.c_str());
    if (v) PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, v);
    Py_XDECREF(v);
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*fn)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<fn, kArgs>)), METH_FASTCALL, nullptr};
}

}  // namespace

PyMODINIT_FUNC PyInit__layer_binding() {
  static PyMethodDef methods[] = {
      {"set_error", set_error, METH_O, nullptr},
      method<conv_fwd, 11>("conv_fwd"),
      method<selective_scan, 15>("selective_scan"),
      method<step, 16>("step"),
      method<w4_matvec, 7>("w4_matvec"),
      method<beam_select, 6>("beam_select"),
      method<beam_reorder, 3>("beam_reorder"),
      method<delta_fwd, 19>("delta_fwd"),
      method<draft_verify, 7>("draft_verify"),
      method<scan_workspace, 5>("scan_workspace"),
      method<select_workspace, 4>("select_workspace"),
      method<delta_workspace, 7>("delta_workspace"),
      method<verify_workspace, 5>("verify_workspace"),
      {nullptr, nullptr, 0, nullptr},
  };
  static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_layer_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&def);
}
