// rollout_ext.cpp -- the Python binding's native half: checks tensors and
// calls the C ABI (include/fp4q/rollout.h), so that a call of a few
// microseconds on the device is not outlasted by its marshalling.  The
// library's entry points are handed over as addresses by bind(); this module
// holds no GPU code and keeps nothing between calls.
#include "ext_common.h"

#include <cmath>

#include "fp4q/rollout.h"

namespace {

decltype(&nvfp4_linear) p_nvfp4_linear;
decltype(&nvfp4_linear_workspace_bytes) p_nvfp4_linear_workspace_bytes;
decltype(&mxfp4_linear) p_mxfp4_linear;
decltype(&mxfp4_linear_workspace_bytes) p_mxfp4_linear_workspace_bytes;
decltype(&nvfp4_kv_append) p_nvfp4_kv_append;
decltype(&nvfp4_kv_read) p_nvfp4_kv_read;
decltype(&nvfp4_kv_attention) p_nvfp4_kv_attention;
decltype(&nvfp4_kv_attention_workspace_bytes) p_nvfp4_kv_attention_workspace_bytes;

// linear(mx, x, codes, scales, row_scales, offsets, fp32, out, workspace) -> out
PyObject* linear(PyObject* const* arg) {
  const bool mx = truth(arg[0]);
  const at::Tensor& x = dense(arg[1], "x", at::kBFloat16);
  const at::Tensor& codes = dense(arg[2], "codes", at::kByte);
  no_gradient(x, "x");
  if (x.dim() != 2) refuse("x must be 2-D [rows, k]");
  const bool grouped = arg[5] != Py_None;
  if (codes.dim() != (grouped ? 3 : 2))
    refuse("codes must be [n, k/2], or [groups, n, k/2] with offsets");
  const int64_t rows = x.size(0), k = x.size(1), n = codes.size(-2);
  const int64_t groups = grouped ? codes.size(0) : 0;
  if (codes.size(-1) * 2 != k)
    refuse("codes hold k = " + std::to_string(codes.size(-1) * 2) + ", x has " +
           std::to_string(k));
  const Device device(x);
  device.same(codes);
  // sizes of the scales, with and without the groups
  const int64_t sizes[] = {groups, n, k / (mx ? 32 : 16)};
  const int64_t* first = grouped ? sizes : sizes + 1;
  const at::Tensor& scales = shaped(arg[3], "scales", at::kByte, {first, sizes + 3});
  device.same(scales);
  const float* row_scales = nullptr;
  if (!mx) {
    const at::Tensor& t = shaped(arg[4], "row_scales", at::kFloat, {first, sizes + 2});
    device.same(t);
    no_gradient(t, "row_scales");
    row_scales = t.const_data_ptr<float>();
  }
  const int64_t* offsets = nullptr;
  if (grouped) {
    const at::Tensor& t = shaped(arg[5], "offsets", at::kLong, {groups + 1});
    device.same(t);
    offsets = t.const_data_ptr<int64_t>();
  }
  bool fp32 = truth(arg[6]);
  at::Tensor out;
  if (arg[7] == Py_None) {
    out = device.empty({rows, n}, fp32 ? at::kFloat : at::kBFloat16);
  } else {
    const at::Tensor& t = tensor(arg[7], "out");
    if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
      refuse(std::string("out must be bfloat16 or float32, got ") + at::toString(t.scalar_type()));
    fp32 = t.scalar_type() == at::kFloat;
    out = shaped(arg[7], "out", t.scalar_type(), {rows, n});
    device.same(out);
  }
  const Workspace ws(arg[8],
                     mx ? p_mxfp4_linear_workspace_bytes(rows, n, k, groups)
                        : p_nvfp4_linear_workspace_bytes(rows, n, k, groups),
                     device);
  const auto* code_bytes = codes.const_data_ptr<uint8_t>();
  const auto* scale_bytes = scales.const_data_ptr<uint8_t>();
  if (mx)
    check(p_mxfp4_linear(x.const_data_ptr(), rows, code_bytes, scale_bytes, n, k, offsets, groups,
                         fp32, out.data_ptr(), ws.data, ws.bytes, device.stream()),
          "mxfp4_linear");
  else
    check(p_nvfp4_linear(x.const_data_ptr(), rows, code_bytes, scale_bytes, row_scales, n, k,
                         offsets, groups, fp32, out.data_ptr(), ws.data, ws.bytes,
                         device.stream()),
          "nvfp4_linear");
  return THPVariable_Wrap(std::move(out));
}

// Holds its six tensors for the length of the call: a sequence may make them as it is read, and
// what the call allocates must not take their memory.
struct Cache {
  struct Held {
    PyObject* p;
    ~Held() { Py_XDECREF(p); }
  } held;
  uint8_t *codes[2], *scales[2];
  float* token_scales[2];
  int64_t pages, heads, page, dim;
  c10::Device device{c10::kCPU};
  Cache(const Cache&) = delete;
  explicit Cache(PyObject* o)
      : held{PySequence_Fast(o, "cache must be an NvFp4KvCache, or its six tensors")} {
    PyObject* seq = held.p;
    if (!seq) throw Raised();
    if (PySequence_Fast_GET_SIZE(seq) != 6)
      refuse("cache must be an NvFp4KvCache, or its six tensors in order");
    PyObject** t = PySequence_Fast_ITEMS(seq);
    const at::Tensor& first = dense(t[0], "k_codes", at::kByte);
    if (first.dim() != 4)
      refuse("k_codes must be 4-D [pages, kv_heads, page_size, head_dim/2]");
    pages = first.size(0), heads = first.size(1), page = first.size(2), dim = 2 * first.size(3);
    device = first.device();
    static const char* const names[] = {"k_codes", "k_scales", "k_token_scales",
                                        "v_codes", "v_scales", "v_token_scales"};
    const Device d(first);
    for (int i = 0; i < 2; ++i) {
      const at::Tensor& c =
          shaped(t[3 * i], names[3 * i], at::kByte, {pages, heads, page, dim / 2});
      // (block scales of values: token innermost)
      const at::Tensor& s = shaped(t[3 * i + 1], names[3 * i + 1], at::kByte,
                                   {pages, heads, i ? dim / 16 : page, i ? page : dim / 16});
      const at::Tensor& f = shaped(t[3 * i + 2], names[3 * i + 2], at::kFloat, {pages, heads, page});
      d.same(c);
      d.same(s);
      d.same(f);
      no_gradient(f, names[3 * i + 2]);
      codes[i] = c.data_ptr<uint8_t>();
      scales[i] = s.data_ptr<uint8_t>();
      token_scales[i] = f.data_ptr<float>();
    }
  }
};

// append(cache, k, v, slots, four_over_six)
PyObject* append(PyObject* const* arg) {
  const Cache c(arg[0]);
  const at::Tensor& k = typed(arg[1], "k", at::kBFloat16);
  const at::Tensor& v = typed(arg[2], "v", at::kBFloat16);
  no_gradient(k, "k");
  no_gradient(v, "v");
  const int64_t ks = token_stride(k, "k", c.heads, c.dim);
  const int64_t vs = token_stride(v, "v", c.heads, c.dim);
  if (k.numel() != v.numel()) refuse("k and v must hold the same tokens");
  const int64_t row = c.heads * c.dim, tokens = row ? k.numel() / row : 0;
  const at::Tensor& slots = sized(arg[3], "slots", at::kLong, tokens);
  const long fos = PyLong_AsLong(arg[4]);
  if (fos == -1 && PyErr_Occurred()) throw Raised();
  const Device device(k);
  device.same(v);
  device.same(slots);
  if (c.device != device.device) refuse("the cache must be on " + device.device.str());
  check(p_nvfp4_kv_append(c.codes[0], c.scales[0], c.token_scales[0], c.codes[1], c.scales[1],
                          c.token_scales[1], c.pages, c.page, c.heads, c.dim, k.const_data_ptr(),
                          ks, v.const_data_ptr(), vs, tokens, slots.const_data_ptr<int64_t>(),
                          (int)fos, device.stream()),
        "nvfp4_kv_append");
  Py_RETURN_NONE;
}

// read(cache, slots, out) -> (k, v)
PyObject* read(PyObject* const* arg) {
  const Cache c(arg[0]);
  const at::Tensor& slots = dense(arg[1], "slots", at::kLong);
  const Device device(slots);
  if (c.device != device.device) refuse("the cache must be on " + device.device.str());
  const int64_t tokens = slots.numel();
  at::Tensor k, v;
  if (arg[2] == Py_None) {
    k = device.empty({tokens, c.heads, c.dim}, at::kBFloat16);
    v = device.empty({tokens, c.heads, c.dim}, at::kBFloat16);
  } else {
    if (!PyTuple_Check(arg[2]) || PyTuple_GET_SIZE(arg[2]) != 2) refuse("out must be (k, v)");
    k = shaped(PyTuple_GET_ITEM(arg[2], 0), "k", at::kBFloat16, {tokens, c.heads, c.dim});
    v = shaped(PyTuple_GET_ITEM(arg[2], 1), "v", at::kBFloat16, {tokens, c.heads, c.dim});
    device.same(k);
    device.same(v);
  }
  check(p_nvfp4_kv_read(c.codes[0], c.scales[0], c.token_scales[0], c.codes[1], c.scales[1],
                        c.token_scales[1], c.pages, c.page, c.heads, c.dim,
                        slots.const_data_ptr<int64_t>(), tokens, k.data_ptr(), v.data_ptr(),
                        device.stream()),
        "nvfp4_kv_read");
  PyObject* a = THPVariable_Wrap(std::move(k));
  PyObject* b = a ? THPVariable_Wrap(std::move(v)) : nullptr;
  PyObject* both = b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return both;
}

// attention(q, cache, page_table, seq_lens, scale, prefix, lse, out, workspace)
//   -> out, or (out, lse)
PyObject* attention(PyObject* const* arg) {
  const at::Tensor& q = typed(arg[0], "q", at::kBFloat16);
  no_gradient(q, "q");
  const Cache c(arg[1]);
  if (q.dim() != 3 && q.dim() != 4)
    refuse("q must be [batch, tokens, heads, head_dim] or [batch, heads, head_dim]");
  const int64_t heads = q.size(-2), batch = q.size(0), tokens = q.dim() == 4 ? q.size(1) : 1;
  const int64_t stride = token_stride(q, "q", heads, c.dim);
  const Device device(q);
  if (c.device != device.device) refuse("the cache must be on " + device.device.str());
  const at::Tensor& table = dense(arg[2], "page_table", at::kInt);
  if (table.dim() != 2 || table.size(0) != batch) refuse("page_table must be [batch, max_pages]");
  const at::Tensor& lens = shaped(arg[3], "seq_lens", at::kInt, {batch});
  device.same(table);
  device.same(lens);
  double scale = 1.0 / std::sqrt((double)c.dim);
  if (arg[4] != Py_None) {
    scale = PyFloat_AsDouble(arg[4]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised();
  }
  const int32_t *ptable = nullptr, *plens = nullptr, *poffsets = nullptr;
  int64_t groups = 0, ppages = 0;
  if (arg[5] != Py_None) {
    if (!PyTuple_Check(arg[5]) || PyTuple_GET_SIZE(arg[5]) != 3)
      refuse("prefix must be (prefix_table, prefix_lens, group_offsets)");
    const at::Tensor& t = dense(PyTuple_GET_ITEM(arg[5], 0), "prefix_table", at::kInt);
    if (t.dim() != 2 || t.size(0) == 0)
      refuse("prefix_table must be [groups, pages] with at least one group");
    groups = t.size(0), ppages = t.size(1);
    const at::Tensor& l = shaped(PyTuple_GET_ITEM(arg[5], 1), "prefix_lens", at::kInt, {groups});
    const at::Tensor& o =
        shaped(PyTuple_GET_ITEM(arg[5], 2), "group_offsets", at::kInt, {groups + 1});
    device.same(t);
    device.same(l);
    device.same(o);
    ptable = t.const_data_ptr<int32_t>();
    plens = l.const_data_ptr<int32_t>();
    poffsets = o.const_data_ptr<int32_t>();
  }
  at::Tensor out;
  if (arg[7] == Py_None) {
    out = device.empty(q.sizes(), at::kBFloat16);
  } else {
    out = shaped(arg[7], "out", at::kBFloat16, q.sizes());
    device.same(out);
  }
  at::Tensor lse;
  if (truth(arg[6])) lse = device.empty(q.sizes().slice(0, q.dim() - 1), at::kFloat);
  const Workspace ws(arg[8],
                     p_nvfp4_kv_attention_workspace_bytes(c.page, c.heads, c.dim, batch, tokens,
                                                          heads, table.size(1), ppages, groups),
                     device);
  check(p_nvfp4_kv_attention(
            c.codes[0], c.scales[0], c.token_scales[0], c.codes[1], c.scales[1],
            c.token_scales[1], c.pages, c.page, c.heads, c.dim, q.const_data_ptr(), stride, batch,
            tokens, heads, table.const_data_ptr<int32_t>(), table.size(1),
            lens.const_data_ptr<int32_t>(), ptable, ppages, plens, poffsets, groups, (float)scale,
            out.data_ptr(), lse.defined() ? lse.data_ptr<float>() : nullptr, ws.data, ws.bytes,
            device.stream()),
        "nvfp4_kv_attention");
  if (!lse.defined()) return THPVariable_Wrap(std::move(out));
  PyObject* a = THPVariable_Wrap(std::move(out));
  PyObject* b = a ? THPVariable_Wrap(std::move(lse)) : nullptr;
  PyObject* both = b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return both;
}

// bind(error type, status check, raw stream getter, eight addresses in the order below)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t count) {
  void* at[8];
  if (!bind_calls(args, count, at)) return nullptr;
  p_nvfp4_linear = (decltype(p_nvfp4_linear))at[0];
  p_nvfp4_linear_workspace_bytes = (decltype(p_nvfp4_linear_workspace_bytes))at[1];
  p_mxfp4_linear = (decltype(p_mxfp4_linear))at[2];
  p_mxfp4_linear_workspace_bytes = (decltype(p_mxfp4_linear_workspace_bytes))at[3];
  p_nvfp4_kv_append = (decltype(p_nvfp4_kv_append))at[4];
  p_nvfp4_kv_read = (decltype(p_nvfp4_kv_read))at[5];
  p_nvfp4_kv_attention = (decltype(p_nvfp4_kv_attention))at[6];
  p_nvfp4_kv_attention_workspace_bytes = (decltype(p_nvfp4_kv_attention_workspace_bytes))at[7];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {FP4Q_METHOD("bind", bind),
                         FP4Q_METHOD("linear", (entry<linear, 9>)),
                         FP4Q_METHOD("append", (entry<append, 5>)),
                         FP4Q_METHOD("read", (entry<read, 3>)),
                         FP4Q_METHOD("attention", (entry<attention, 9>)),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "fp4q_rollout_ext", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fp4q_rollout_ext() { return PyModule_Create(&module); }
