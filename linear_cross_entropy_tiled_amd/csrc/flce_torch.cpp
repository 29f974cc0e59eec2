// The PyTorch side of layer_norm and embedding, operators whose autograd nodes are C++, and
// of the MXFP4 calls.  The Python functions in front of them (norm.py, embedding.py,
// logprobs.py) check arguments and say what is wrong with them; types, sizes, layout and
// device, which the kernels trust, are checked here again, since a recorded graph calls
// these operators without Python, with tensors other than the recorded ones.  The work is
// that of the C ABI, whose entry points are handed over by address once, so that this
// library runs on whichever build of libflce.so is loaded.
//
// Why not a Python autograd function, as the other operators have: autograd runs a GPU
// node's backward on a thread of its own, and Python that wakes up there runs at half its
// speed.  A layer norm training step of 515 x 1023 took 115 us that way and takes 76 so, of which 15 are the GPU's.
// The MXFP4 calls have no node; their few microseconds of GPU time wait for allocations and argument lists in Python
// (250 x 4096 values to 4 bits and back: 18.7 us, 7 of them the GPU's).
#include <ATen/ATen.h>
#include <ATen/hip/impl/HIPGuardImplMasqueradingAsCUDA.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/library.h>

#include <optional>
#include <tuple>

#include "../../include/flce.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

struct EntryPoints {
  decltype(&flce_layer_norm_forward) norm_forward = nullptr;
  decltype(&flce_layer_norm_backward) norm_backward = nullptr;
  decltype(&flce_embedding_forward) embedding_forward = nullptr;
  decltype(&flce_embedding_backward) embedding_backward = nullptr;
  decltype(&flce_quantize_mxfp4) quantize = nullptr;
  decltype(&flce_dequantize_mxfp4) dequantize = nullptr;
  decltype(&flce_logprobs_mxfp4) scores = nullptr;
  decltype(&flce_status_string) status_string = nullptr;
} g;

void bind(at::IntArrayRef at) {
  TORCH_CHECK(at.size() == 8, "eight entry points are expected");
  g.norm_forward = reinterpret_cast<decltype(g.norm_forward)>(at[0]);
  g.norm_backward = reinterpret_cast<decltype(g.norm_backward)>(at[1]);
  g.embedding_forward = reinterpret_cast<decltype(g.embedding_forward)>(at[2]);
  g.embedding_backward = reinterpret_cast<decltype(g.embedding_backward)>(at[3]);
  g.quantize = reinterpret_cast<decltype(g.quantize)>(at[4]);
  g.dequantize = reinterpret_cast<decltype(g.dequantize)>(at[5]);
  g.scores = reinterpret_cast<decltype(g.scores)>(at[6]);
  g.status_string = reinterpret_cast<decltype(g.status_string)>(at[7]);
}

void ok(int rc, const char* where) {
  TORCH_CHECK(rc == FLCE_OK, where, ": ", g.status_string(rc), " (", rc, ")");
}

bool is_value(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16 || t == at::kHalf; }
bool is_id(const Tensor& t) { return t.scalar_type() == at::kLong || t.scalar_type() == at::kInt; }
// A contiguous tensor of these sizes, on the GPU of `first`.
bool is_whole(const Tensor& t, at::IntArrayRef sizes, const Tensor& first) {
  return t.sizes() == sizes && t.is_contiguous() && t.is_cuda() && t.device() == first.device();
}
bool is_codes(const Tensor& q, const Tensor& scale, const Tensor& first) {
  return q.dim() == 2 && q.size(1) > 0 && q.size(1) % 16 == 0 && q.scalar_type() == at::kByte &&
         is_whole(q, q.sizes(), first) && scale.scalar_type() == at::kByte &&
         is_whole(scale, {q.size(0), q.size(1) / 16}, first);
}
void expect(bool taken, const char* where) {
  TORCH_CHECK(taken, where, ": a tensor of a type, size, layout or device that this call does not take");
}

int32_t type_of(const Tensor& t) {
  return t.scalar_type() == at::kFloat ? FLCE_F32 : (t.scalar_type() == at::kBFloat16 ? FLCE_BF16 : FLCE_F16);
}
void* data(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
void* stream_of(const Tensor& t) {
  return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(t.device().index()).stream();
}
using Guard = c10::hip::HIPGuardMasqueradingAsCUDA;   // the library launches on the current device

// Rows that are contiguous and do not overlap, at any distance.
bool rows_apart(const Tensor& t) {
  return t.is_contiguous() || ((t.stride(1) == 1 || t.size(1) == 1) && (t.stride(0) >= t.size(1) || t.size(0) == 1));
}
int64_t row_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// Gradients without a derivative of their own: taking one raises.
variable_list first_order(variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  for (auto& t : grads)
    if (t.defined()) t = t.detach().set_requires_grad(true);
  const auto error = std::make_shared<torch::autograd::DelayedError>("this gradient has no derivative of its own",
                                                                     (int64_t)grads.size());
  return (*error)(std::move(grads));
}

// ----------------------------------------------------------------------------- layer norm

flce_norm_params norm_params(const Tensor& x, const Tensor& weight, const Tensor& bias, double eps) {
  flce_norm_params p{};
  p.rows = x.size(0);
  p.cols = x.size(1);
  p.ld_x = row_stride(x);
  p.dtype = type_of(x);
  p.param_dtype = weight.defined() ? type_of(weight) : (bias.defined() ? type_of(bias) : p.dtype);
  p.eps = (float)eps;
  return p;
}

// stats: [2][rows] fp32, or undefined where no backward follows.
Tensor norm_forward(const Tensor& x, const Tensor& weight, const Tensor& bias, double eps, const Tensor& stats) {
  const flce_norm_params p = norm_params(x, weight, bias, eps);
  Tensor y = at::empty({p.rows, p.cols}, x.options());
  float* mean = stats.defined() ? stats.data_ptr<float>() : nullptr;
  ok(g.norm_forward(&p, data(x), data(weight), data(bias), data(y), mean, mean ? mean + p.rows : nullptr, stream_of(x)),
     "flce_layer_norm_forward");
  return y;
}

struct LayerNorm : torch::autograd::Function<LayerNorm> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const std::optional<Tensor>& weight,
                        const std::optional<Tensor>& bias, double eps, int64_t workspace) {
    const Guard guard(x.device());
    const Tensor w = weight.value_or(Tensor()), b = bias.value_or(Tensor());
    const Tensor stats = at::empty({2, x.size(0)}, x.options().dtype(at::kFloat));
    ctx->save_for_backward({x, w, b, stats});
    ctx->saved_data["eps"] = eps;
    ctx->saved_data["workspace"] = workspace;
    return norm_forward(x, w, b, eps, stats);
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &x = saved[0], &w = saved[1], &b = saved[2], &stats = saved[3];
    const Guard guard(x.device());
    const Tensor dy = rows_apart(grads[0]) ? grads[0] : grads[0].contiguous();
    flce_norm_params p = norm_params(x, w, b, ctx->saved_data["eps"].toDouble());
    p.ld_grad = row_stride(dy);
    Tensor dx, dw, db, workspace;
    // the gradients that this backward was asked for; inputs are counted without absent ones
    if (ctx->needs_input_grad(0)) dx = at::empty({p.rows, p.cols}, x.options());
    if (w.defined() && ctx->needs_input_grad(1)) dw = at::empty({p.cols}, w.options());
    if (b.defined() && ctx->needs_input_grad(w.defined() ? 2 : 1)) db = at::empty({p.cols}, b.options());
    const int64_t bytes = dw.defined() || db.defined() ? ctx->saved_data["workspace"].toInt() : 0;
    if (bytes > 0) workspace = at::empty({bytes}, x.options().dtype(at::kByte));
    const float* mean = stats.data_ptr<float>();
    ok(g.norm_backward(&p, data(x), data(w), mean, mean ? mean + p.rows : nullptr, data(dy), data(dx), data(dw), data(db),
                       data(workspace), (size_t)bytes, stream_of(x)),
       "flce_layer_norm_backward");
    return first_order({dx, dw, db, Tensor(), Tensor()});
  }
};

bool is_param(const std::optional<Tensor>& t, const Tensor& x) {
  return !t || !t->defined() ||
         ((t->scalar_type() == x.scalar_type() || t->scalar_type() == at::kFloat) && is_whole(*t, {x.size(1)}, x));
}

Tensor layer_norm(const Tensor& x, const std::optional<Tensor>& weight, const std::optional<Tensor>& bias, double eps,
                  int64_t workspace) {
  const bool both = weight && weight->defined() && bias && bias->defined();
  expect(x.dim() == 2 && x.size(1) > 0 && is_value(x.scalar_type()) && x.is_cuda() && rows_apart(x) &&
             is_param(weight, x) && is_param(bias, x) && (!both || weight->scalar_type() == bias->scalar_type()),
         "layer_norm");
  const auto recorded = [](const std::optional<Tensor>& t) { return t && t->defined() && t->requires_grad(); };
  if (at::GradMode::is_enabled() && (x.requires_grad() || recorded(weight) || recorded(bias)))
    return LayerNorm::apply(x, weight, bias, eps, workspace);
  const Guard guard(x.device());
  return norm_forward(x, weight.value_or(Tensor()), bias.value_or(Tensor()), eps, Tensor());
}

// ----------------------------------------------------------------------------- embedding

flce_embedding_params embedding_params(const Tensor& ids, const Tensor& rows, int64_t vocab, double scale,
                                       int64_t ignore_index) {
  flce_embedding_params p{};
  p.n_tokens = ids.size(0);
  p.hidden = rows.size(1);
  p.vocab = vocab;
  p.ignore_index = ignore_index;
  p.dtype = p.grad_weight_dtype = type_of(rows);
  p.flags = ids.scalar_type() == at::kInt ? FLCE_TARGETS_INT32 : 0;
  p.scale = (float)scale;
  return p;
}

Tensor embedding_forward(const Tensor& ids, const Tensor& weight, double scale, int64_t ignore_index) {
  const Guard guard(weight.device());
  const flce_embedding_params p = embedding_params(ids, weight, weight.size(0), scale, ignore_index);
  Tensor out = at::empty({p.n_tokens, p.hidden}, weight.options());
  ok(g.embedding_forward(&p, data(ids), data(weight), data(out), stream_of(weight)), "flce_embedding_forward");
  return out;
}

struct Embedding : torch::autograd::Function<Embedding> {
  static Tensor forward(AutogradContext* ctx, const Tensor& weight, const Tensor& ids, double scale,
                        int64_t ignore_index, int64_t workspace) {
    ctx->save_for_backward({ids});
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["ignore_index"] = ignore_index;
    ctx->saved_data["vocab"] = weight.size(0);
    ctx->saved_data["workspace"] = workspace;
    return embedding_forward(ids, weight, scale, ignore_index);
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const Tensor ids = ctx->get_saved_variables()[0], dy = grads[0].contiguous();
    const Guard guard(dy.device());
    const int64_t bytes = ctx->saved_data["workspace"].toInt();
    const flce_embedding_params p =
        embedding_params(ids, dy, ctx->saved_data["vocab"].toInt(), ctx->saved_data["scale"].toDouble(),
                         ctx->saved_data["ignore_index"].toInt());
    const Tensor dw = at::empty({p.vocab, p.hidden}, dy.options());
    const Tensor workspace = at::empty({bytes}, dy.options().dtype(at::kByte));
    ok(g.embedding_backward(&p, data(ids), data(dy), data(dw), data(workspace), (size_t)bytes, stream_of(dy)),
       "flce_embedding_backward");
    return first_order({dw, Tensor(), Tensor(), Tensor(), Tensor()});
  }
};

Tensor embedding(const Tensor& ids, const Tensor& weight, double scale, int64_t ignore_index, int64_t workspace) {
  expect(ids.dim() == 1 && is_id(ids) && is_whole(ids, ids.sizes(), weight) && weight.dim() == 2 && weight.size(0) > 0 &&
             weight.size(1) > 0 && is_value(weight.scalar_type()) && is_whole(weight, weight.sizes(), weight),
         "embedding");
  if (at::GradMode::is_enabled() && weight.requires_grad())
    return Embedding::apply(weight, ids, scale, ignore_index, workspace);
  return embedding_forward(ids, weight, scale, ignore_index);
}

// ----------------------------------------------------------------------------- MXFP4

std::tuple<Tensor, Tensor> quantize_mxfp4(const Tensor& x) {
  expect(x.dim() == 2 && x.size(1) > 0 && x.size(1) % 32 == 0 && is_value(x.scalar_type()) && is_whole(x, x.sizes(), x),
         "quantize_mxfp4");
  const Guard guard(x.device());
  const int64_t rows = x.size(0), cols = x.size(1);
  const auto bytes = x.options().dtype(at::kByte).requires_grad(false);
  const Tensor q = at::empty({rows, cols / 2}, bytes), scale = at::empty({rows, cols / 32}, bytes);
  ok(g.quantize(type_of(x), data(x), rows, cols, data(q), data(scale), stream_of(x)), "flce_quantize_mxfp4");
  return {q, scale};
}

Tensor dequantize_mxfp4(const Tensor& q, const Tensor& scale, at::ScalarType dtype) {
  expect(is_codes(q, scale, q) && is_value(dtype), "dequantize_mxfp4");
  const Guard guard(q.device());
  const int64_t rows = q.size(0), cols = 2 * q.size(1);
  const Tensor x = at::empty({rows, cols}, q.options().dtype(dtype));
  ok(g.dequantize(type_of(x), data(q), data(scale), rows, cols, data(x), stream_of(q)), "flce_dequantize_mxfp4");
  return x;
}

// workspace: its bytes.  hidden without scales holds values.  The entropies are undefined where they are not wanted.
std::tuple<Tensor, Tensor> logprobs_mxfp4(const Tensor& hidden, const std::optional<Tensor>& hidden_scale,
                                          const Tensor& weight, const Tensor& weight_scale,
                                          const std::optional<Tensor>& bias, const Tensor& targets, double logit_scale,
                                          double softcap, int64_t ignore_index, int64_t workspace, bool want_entropy) {
  expect(is_codes(weight, weight_scale, hidden) && hidden.dim() == 2 &&
             (hidden_scale ? is_codes(hidden, *hidden_scale, hidden) && hidden.size(1) == weight.size(1)
                           : is_value(hidden.scalar_type()) &&
                                 is_whole(hidden, {hidden.size(0), 2 * weight.size(1)}, hidden)) &&
             is_id(targets) && is_whole(targets, {hidden.size(0)}, hidden) &&
             (!bias || (bias->scalar_type() == at::kFloat && is_whole(*bias, {weight.size(0)}, hidden))),
         "token_logprobs_mxfp4");
  const Guard guard(hidden.device());
  const int64_t n = hidden.size(0);
  flce_params p{};
  p.n_tokens = n;
  p.hidden = 2 * weight.size(1);
  p.vocab = weight.size(0);
  p.ignore_index = ignore_index;
  p.dtype = p.grad_weight_dtype = hidden_scale ? FLCE_BF16 : type_of(hidden);
  p.reduction = FLCE_REDUCTION_NONE;
  p.flags = targets.scalar_type() == at::kInt ? FLCE_TARGETS_INT32 : 0;
  p.logit_scale = (float)logit_scale;
  p.softcap = (float)softcap;
  const auto floats = weight.options().dtype(at::kFloat);
  // one allocation: the workspace, then the log-sum-exps, which nobody asked for
  const Tensor room = at::empty({workspace + 4 * n}, weight.options()), logps = at::empty({n}, floats);
  Tensor entropy;
  if (want_entropy) entropy = at::empty({n}, floats);
  char* at = static_cast<char*>(data(room));
  ok(g.scores(&p, data(hidden), data(hidden_scale.value_or(Tensor())), data(weight), data(weight_scale),
              static_cast<const float*>(data(bias.value_or(Tensor()))), data(targets), static_cast<float*>(data(logps)),
              static_cast<float*>(data(entropy)), reinterpret_cast<float*>(at + workspace), at, (size_t)workspace,
              stream_of(hidden)),
     "flce_logprobs_mxfp4");
  return {logps, entropy};
}

}  // namespace

TORCH_LIBRARY(flce, m) {
  m.def("_bind(int[] entry_points) -> ()", bind);
  m.def("_layer_norm(Tensor x, Tensor? weight, Tensor? bias, float eps, int workspace) -> Tensor", layer_norm);
  m.def("_quantize_mxfp4(Tensor x) -> (Tensor, Tensor)", quantize_mxfp4);
  m.def("_dequantize_mxfp4(Tensor q, Tensor scale, ScalarType dtype) -> Tensor", dequantize_mxfp4);
  m.def(
      "_logprobs_mxfp4(Tensor hidden, Tensor? hidden_scale, Tensor weight, Tensor weight_scale, Tensor? bias, "
      "Tensor targets, float logit_scale, float softcap, int ignore_index, int workspace, bool entropy) -> "
      "(Tensor, Tensor)",
      logprobs_mxfp4);
  m.def("_embedding(Tensor ids, Tensor weight, float scale, int ignore_index, int workspace) -> Tensor", embedding);
}
