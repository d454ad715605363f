// layer_ext.cpp -- the Python binding's native half for the operators of
// include/fp4q/layer.h: checks tensors and calls the C ABI, in the manner of
// rollout_ext.cpp.  The library's entry points are handed over as addresses
// by bind(); this module holds no GPU code and keeps nothing between calls.
#include "ext_common.h"

#include <cmath>

#include "fp4q/layer.h"

namespace {

decltype(&rotary_embed) p_rotary_embed;
decltype(&prompt_attention) p_prompt_attention;
decltype(&prompt_attention_workspace_bytes) p_prompt_attention_workspace_bytes;
decltype(&moe_route) p_moe_route;
decltype(&moe_dispatch) p_moe_dispatch;
decltype(&moe_dispatch_workspace_bytes) p_moe_dispatch_workspace_bytes;
decltype(&moe_combine) p_moe_combine;

// Sizes that outputs are allocated by, refused here before that.
constexpr int64_t kMaxChoices = 64, kMaxExperts = 1024;

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

// BF16 or FP32, which the second says.
const at::Tensor& either(PyObject* o, const char* name, bool& fp32) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
    refuse(std::string(name) + " must be bfloat16 or float32, got " +
           at::toString(t.scalar_type()));
  fp32 = t.scalar_type() == at::kFloat;
  return t;
}

PyObject* wrapped(at::Tensor* t, Py_ssize_t n) {
  PyObject* all = PyTuple_New(n);
  if (!all) return nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = Py_None;
    if (t[i].defined())
      o = THPVariable_Wrap(std::move(t[i]));
    else
      Py_INCREF(o);
    if (!o) {
      Py_DECREF(all);
      return nullptr;
    }
    PyTuple_SET_ITEM(all, i, o);
  }
  return all;
}

// The parts of an out=(..) argument.
PyObject** parts_of(PyObject* out, Py_ssize_t n, const char* what) {
  if (!PyTuple_Check(out) || PyTuple_GET_SIZE(out) != n) refuse(std::string("out must be ") + what);
  return ((PyTupleObject*)out)->ob_item;
}

// rotary(q, k, positions, frequencies, amplitude, interleaved, inverse, out) -> (q, k)
PyObject* rotary(PyObject* const* arg) {
  bool fp32 = false;
  const at::Tensor* in[2] = {&either(arg[0], "q", fp32), nullptr};
  if (in[0]->dim() < 3) refuse("q must be [..., heads, head_dim]");
  const at::ScalarType type = in[0]->scalar_type();
  const Device device(*in[0]);
  if (arg[1] != Py_None) {
    in[1] = &typed(arg[1], "k", type);
    if (in[1]->dim() < 3) refuse("k must be [..., heads, head_dim]");
    device.same(*in[1]);
  }
  static const char* const names[] = {"q", "k"};
  static const char* const out_names[] = {"q's out", "k's out"};
  const int64_t dim = in[0]->size(-1);
  PyObject** given = arg[7] == Py_None ? nullptr : parts_of(arg[7], 2, "(q, k)");
  int64_t heads[2] = {0, 0}, stride[2] = {0, 0}, out_stride[2] = {0, 0}, tokens = 0;
  at::Tensor out[2];
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) {
      if (given && given[i] != Py_None) refuse("out has a tensor for k, which is None");
      continue;
    }
    const at::Tensor& t = *in[i];
    no_gradient(t, names[i]);
    heads[i] = t.size(-2);
    stride[i] = token_stride(t, names[i], heads[i], dim);
    int64_t n = 1;
    for (int64_t j = 0; j < t.dim() - 2; ++j) n *= t.size(j);
    if (i == 0)
      tokens = n;
    else if (n != tokens)
      refuse("q and k must hold the same tokens");
    if (given) {
      out[i] = typed(given[i], out_names[i], type);
      if (out[i].sizes() != t.sizes())
        refuse(std::string(out_names[i]) + " must be " + text_of(t.sizes()) + ", got " +
               text_of(out[i].sizes()));
      device.same(out[i]);
      no_gradient(out[i], out_names[i]);
      out_stride[i] = token_stride(out[i], out_names[i], heads[i], dim);
    } else {
      out_stride[i] = heads[i] * dim;
    }
  }
  if (!given && in[1])
    allocate(device, {in[0]->sizes(), in[1]->sizes()}, {type, type}, out);
  else if (!given)
    out[0] = device.empty(in[0]->sizes(), type);
  const at::Tensor& positions = sized(arg[2], "positions", at::kLong, tokens);
  const at::Tensor& frequencies = dense(arg[3], "frequencies", at::kDouble);
  if (frequencies.dim() != 1) refuse("frequencies must be [dims / 2]");
  device.same(positions);
  device.same(frequencies);
  no_gradient(frequencies, "frequencies");
  const double amplitude = real(arg[4]);
  check(p_rotary_embed(in[0]->const_data_ptr(), stride[0], heads[0],
                       in[1] ? in[1]->const_data_ptr() : nullptr, stride[1], heads[1], tokens, dim,
                       2 * frequencies.numel(), positions.const_data_ptr<int64_t>(),
                       frequencies.const_data_ptr<double>(), (float)amplitude, truth(arg[5]),
                       truth(arg[6]), fp32, out[0].data_ptr(), out_stride[0],
                       out[1].defined() ? out[1].data_ptr() : nullptr, out_stride[1],
                       device.stream()),
        "rotary_embed");
  return wrapped(out, 2);
}

// prompt(q, k, v, q_offsets, k_offsets, scale, lse, out, workspace) -> out, or (out, lse)
PyObject* prompt(PyObject* const* arg) {
  const at::Tensor& q = typed(arg[0], "q", at::kBFloat16);
  const at::Tensor& k = typed(arg[1], "k", at::kBFloat16);
  const at::Tensor& v = typed(arg[2], "v", at::kBFloat16);
  no_gradient(q, "q");
  no_gradient(k, "k");
  no_gradient(v, "v");
  if (q.dim() != 3 || k.dim() != 3 || v.dim() != 3)
    refuse("q, k and v must be [tokens, heads, head_dim]");
  const int64_t q_tokens = q.size(0), heads = q.size(1), dim = q.size(2);
  const int64_t k_tokens = k.size(0), kv_heads = k.size(1);
  if (v.size(0) != k_tokens) refuse("k and v must hold the same tokens");
  const int64_t qs = token_stride(q, "q", heads, dim);
  const int64_t ks = token_stride(k, "k", kv_heads, dim);
  const int64_t vs = token_stride(v, "v", kv_heads, dim);
  const Device device(q);
  device.same(k);
  device.same(v);
  const at::Tensor& q_off = dense(arg[3], "q_offsets", at::kInt);
  if (q_off.dim() != 1 || q_off.numel() == 0) refuse("q_offsets must be [sequences + 1]");
  device.same(q_off);
  const int64_t batch = q_off.numel() - 1;
  const at::Tensor& k_off =
      arg[4] == Py_None ? q_off : shaped(arg[4], "k_offsets", at::kInt, {batch + 1});
  device.same(k_off);
  const double scale = arg[5] == Py_None ? 1.0 / std::sqrt((double)dim) : real(arg[5]);
  at::Tensor out[2];
  const bool lse = truth(arg[6]);
  const int64_t lse_shape[] = {q_tokens, heads};
  if (arg[7] == Py_None && lse) {
    allocate(device, {q.sizes(), lse_shape}, {at::kBFloat16, at::kFloat}, out);
  } else if (arg[7] == Py_None) {
    out[0] = device.empty(q.sizes(), at::kBFloat16);
  } else {
    out[0] = shaped(arg[7], "out", at::kBFloat16, q.sizes());
    device.same(out[0]);
    no_gradient(out[0], "out");
  }
  if (lse && !out[1].defined()) out[1] = device.empty(lse_shape, at::kFloat);
  const Workspace ws(
      arg[8],
      p_prompt_attention_workspace_bytes(q_tokens, heads, k_tokens, kv_heads, dim, batch), device);
  check(p_prompt_attention(q.const_data_ptr(), qs, q_tokens, heads, k.const_data_ptr(), ks,
                           v.const_data_ptr(), vs, k_tokens, kv_heads, dim,
                           q_off.const_data_ptr<int32_t>(), k_off.const_data_ptr<int32_t>(), batch,
                           (float)scale, out[0].data_ptr(),
                           out[1].defined() ? out[1].data_ptr<float>() : nullptr, ws.data, ws.bytes,
                           device.stream()),
        "prompt_attention");
  return out[1].defined() ? wrapped(out, 2) : THPVariable_Wrap(std::move(out[0]));
}

// route(logits, top_k, bias, scoring, groups, top_groups, renormalize, scale, active, out)
//   -> (weights, experts)
PyObject* route(PyObject* const* arg) {
  bool fp32 = false;
  const at::Tensor& logits = either(arg[0], "logits", fp32);
  if (logits.dim() != 2 || !logits.is_contiguous())
    refuse("logits must be a contiguous [tokens, experts]");
  no_gradient(logits, "logits");
  const int64_t tokens = logits.size(0), experts = logits.size(1), top_k = integer(arg[1]);
  const Device device(logits);
  const float* bias = nullptr;
  if (arg[2] != Py_None) {
    const at::Tensor& t = shaped(arg[2], "bias", at::kFloat, {experts});
    device.same(t);
    no_gradient(t, "bias");
    bias = t.const_data_ptr<float>();
  }
  const uint8_t* active = nullptr;
  if (arg[8] != Py_None) {
    const at::Tensor& t = shaped(arg[8], "active", at::kBool, {tokens});
    device.same(t);
    active = (const uint8_t*)t.const_data_ptr();
  }
  if (top_k < 1 || top_k > kMaxChoices)
    refuse("top_k must be 1 to " + std::to_string(kMaxChoices));
  at::Tensor out[2];
  if (arg[9] == Py_None) {
    const int64_t shape[] = {tokens, top_k};
    allocate(device, {shape, shape}, {at::kFloat, at::kInt}, out);
  } else {
    PyObject** given = parts_of(arg[9], 2, "(weights, experts)");
    out[0] = shaped(given[0], "weights", at::kFloat, {tokens, top_k});
    out[1] = shaped(given[1], "experts", at::kInt, {tokens, top_k});
    device.same(out[0]);
    device.same(out[1]);
    no_gradient(out[0], "weights");
  }
  check(p_moe_route(logits.const_data_ptr(), fp32, tokens, experts, top_k, bias,
                    (int)integer(arg[3]), integer(arg[4]), integer(arg[5]), truth(arg[6]),
                    (float)real(arg[7]), active, out[0].data_ptr<float>(),
                    out[1].data_ptr<int32_t>(), device.stream()),
        "moe_route");
  return wrapped(out, 2);
}

// dispatch(x, experts, num_experts, out, workspace) -> (rows, offsets, place)
PyObject* dispatch(PyObject* const* arg) {
  const at::Tensor& x = dense(arg[0], "x", at::kBFloat16);
  const at::Tensor& chosen = dense(arg[1], "experts", at::kInt);
  no_gradient(x, "x");
  if (x.dim() != 2) refuse("x must be 2-D [tokens, hidden]");
  if (chosen.dim() != 2 || chosen.size(0) != x.size(0)) refuse("experts must be [tokens, top_k]");
  const int64_t tokens = x.size(0), hidden = x.size(1), top_k = chosen.size(1);
  const int64_t experts = integer(arg[2]);
  if (experts < 1 || experts > kMaxExperts)
    refuse("num_experts must be 1 to " + std::to_string(kMaxExperts));
  const Device device(x);
  device.same(chosen);
  at::Tensor out[3];
  if (arg[3] == Py_None) {
    const int64_t offsets[] = {experts + 1}, place[] = {tokens, top_k};
    out[0] = device.empty({tokens * top_k, hidden}, at::kBFloat16);
    allocate(device, {offsets, place}, {at::kLong, at::kInt}, out + 1);
  } else {
    PyObject** given = parts_of(arg[3], 3, "(rows, offsets, place)");
    out[0] = shaped(given[0], "rows", at::kBFloat16, {tokens * top_k, hidden});
    out[1] = shaped(given[1], "offsets", at::kLong, {experts + 1});
    out[2] = shaped(given[2], "place", at::kInt, {tokens, top_k});
    for (const at::Tensor& t : out) device.same(t);
    no_gradient(out[0], "rows");
  }
  const Workspace ws(arg[4], p_moe_dispatch_workspace_bytes(tokens, top_k, experts), device);
  check(p_moe_dispatch(x.const_data_ptr(), tokens, hidden, chosen.const_data_ptr<int32_t>(), top_k,
                       experts, out[0].data_ptr(), out[1].data_ptr<int64_t>(),
                       out[2].data_ptr<int32_t>(), ws.data, ws.bytes, device.stream()),
        "moe_dispatch");
  return wrapped(out, 3);
}

// combine(y, place, weights, add, fp32, out) -> out
PyObject* combine(PyObject* const* arg) {
  bool y_fp32 = false;
  const at::Tensor& y = either(arg[0], "y", y_fp32);
  if (y.dim() != 2 || !y.is_contiguous()) refuse("y must be a contiguous [rows, n]");
  no_gradient(y, "y");
  const at::Tensor& place = dense(arg[1], "place", at::kInt);
  if (place.dim() != 2) refuse("place must be [tokens, top_k]");
  const int64_t tokens = place.size(0), top_k = place.size(1), n = y.size(1);
  const at::Tensor& weights = shaped(arg[2], "weights", at::kFloat, {tokens, top_k});
  no_gradient(weights, "weights");
  const Device device(y);
  device.same(place);
  device.same(weights);
  const void* add = nullptr;
  if (arg[3] != Py_None) {
    const at::Tensor& t = shaped(arg[3], "add", at::kBFloat16, {tokens, n});
    device.same(t);
    no_gradient(t, "add");
    add = t.const_data_ptr();
  }
  bool fp32 = truth(arg[4]);
  at::Tensor out;
  if (arg[5] == Py_None) {
    out = device.empty({tokens, n}, fp32 ? at::kFloat : at::kBFloat16);
  } else {
    const at::Tensor& t = either(arg[5], "out", fp32);
    out = shaped(arg[5], "out", t.scalar_type(), {tokens, n});
    device.same(out);
    no_gradient(out, "out");
  }
  check(p_moe_combine(y.const_data_ptr(), y_fp32, y.size(0), place.const_data_ptr<int32_t>(),
                      weights.const_data_ptr<float>(), add, tokens, top_k, n, fp32, out.data_ptr(),
                      device.stream()),
        "moe_combine");
  return THPVariable_Wrap(std::move(out));
}

// bind(error type, status check, raw stream getter, seven addresses in the order below)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t count) {
  void* at[7];
  if (!bind_calls(args, count, at)) return nullptr;
  p_rotary_embed = (decltype(p_rotary_embed))at[0];
  p_prompt_attention = (decltype(p_prompt_attention))at[1];
  p_prompt_attention_workspace_bytes = (decltype(p_prompt_attention_workspace_bytes))at[2];
  p_moe_route = (decltype(p_moe_route))at[3];
  p_moe_dispatch = (decltype(p_moe_dispatch))at[4];
  p_moe_dispatch_workspace_bytes = (decltype(p_moe_dispatch_workspace_bytes))at[5];
  p_moe_combine = (decltype(p_moe_combine))at[6];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {FP4Q_METHOD("bind", bind),
                         FP4Q_METHOD("rotary", (entry<rotary, 8>)),
                         FP4Q_METHOD("prompt", (entry<prompt, 9>)),
                         FP4Q_METHOD("route", (entry<route, 10>)),
                         FP4Q_METHOD("dispatch", (entry<dispatch, 5>)),
                         FP4Q_METHOD("combine", (entry<combine, 6>)),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "fp4q_layer_ext", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fp4q_layer_ext() { return PyModule_Create(&module); }
