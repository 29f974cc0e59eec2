// C ABI of the preference and policy losses: argument validation, the split of
// the tokens over waves, workspace layout.  Validation runs on the host before
// any HIP call.
#include <math.h>
#include <string.h>

#include "flce_align.h"

namespace flce {

// Waves a pass over the tokens aims for: 32 a CU.  With 16 the full policy loss over
// 2048 x 8192 tokens took 154 us forward and backward, with 32 it takes 146 (4.4 TB/s of
// the 4.7 of a large copy), with 64 151; at 2048 x 2048 all three are within 3%.
static constexpr int64_t kTargetWaves = 8192;
static constexpr int64_t kMaxSeqs = int64_t(1) << 24;
static constexpr int64_t kMaxTokens = int64_t(1) << 40;

static bool align_dtype_ok(int d) { return d == FLCE_F32 || d == FLCE_BF16 || d == FLCE_F16; }
static size_t align256(size_t x) { return (x + 255) / 256 * 256; }

static int plan_seqs(int64_t S, int64_t length, bool packed, Seqs* q) {
  memset(q, 0, sizeof(*q));
  if (S < 0 || length < 0) return FLCE_ERR_INVALID_ARG;
  if (S > kMaxSeqs || length > kMaxTokens) return FLCE_ERR_UNSUPPORTED;
  if (!packed && S > 0 && length > kMaxTokens / S) return FLCE_ERR_UNSUPPORTED;
  const int64_t tokens = packed ? length : S * length;
  const int64_t steps = (tokens + 256 * kTargetWaves - 1) / (256 * kTargetWaves);
  q->S = S;
  q->length = length;
  q->packed = packed ? 1 : 0;
  q->chunk = 256 * (steps > 1 ? steps : 1);
  q->chunks_per_row = (length + q->chunk - 1) / q->chunk;
  q->waves = packed ? q->chunks_per_row : S * q->chunks_per_row;
  return FLCE_OK;
}

static int64_t slot_count(const Seqs& q) { return q.waves + (q.packed ? q.S : 0); }

// Lanes that add one sequence's slots, a power of two: four slots to a lane on average,
// whose loads it has in flight together.
static int slot_group(const Seqs& q) {
  const int64_t each = q.S > 0 ? (q.waves + q.S - 1) / q.S : 1;
  int g = 1;
  while (g < 64 && 4 * g < each) g *= 2;
  return g;
}

static int64_t max_slots(int64_t S, int64_t length, int* rc) {
  Seqs a, b;
  *rc = plan_seqs(S, length, false, &a);
  if (*rc != FLCE_OK) return 0;
  *rc = plan_seqs(S, length, true, &b);
  if (*rc != FLCE_OK) return 0;
  const int64_t x = slot_count(a), y = slot_count(b);
  return x > y ? x : y;
}

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// One token tensor: its stride, and whether rows of it can be read four elements at a time.
static int check_view(const flce_token_view& v, const Seqs& q, size_t esize, int64_t* ld, bool* vec) {
  if (!v.data) {
    *ld = 0;
    return FLCE_OK;
  }
  if (!aligned(v.data, esize)) return FLCE_ERR_UNSUPPORTED;
  *ld = q.packed || v.ld == 0 ? q.length : v.ld;
  if (*ld < q.length) return FLCE_ERR_INVALID_ARG;
  if (!aligned(v.data, 4 * esize) || (!q.packed && *ld % 4 != 0)) *vec = false;
  return FLCE_OK;
}

static int check_layout(const flce_token_view& mask, const void* offsets, int flags, Seqs* q, bool* vec) {
  q->offsets = offsets;
  q->off_i32 = (flags & FLCE_OFFSETS_INT32) ? 1 : 0;
  if (offsets && !aligned(offsets, q->off_i32 ? 4 : 8)) return FLCE_ERR_UNSUPPORTED;
  q->mask = static_cast<const uint8_t*>(mask.data);
  if (!q->packed && q->length % 4 != 0) *vec = false;   // rows of the contiguous outputs
  return check_view(mask, *q, 1, &q->ld_mask, vec);
}

static size_t esize_of(int dtype) { return dtype == FLCE_F32 ? 4 : 2; }

static int check_preference(const flce_preference_params* p) {
  if (!p || p->n_seqs < 0 || p->n_seqs % 2 != 0 || p->length < 0) return FLCE_ERR_INVALID_ARG;
  if (!align_dtype_ok(p->dtype) || p->type < FLCE_PREFERENCE_SIGMOID || p->type > FLCE_PREFERENCE_SQUARED)
    return FLCE_ERR_INVALID_ARG;
  if (p->reduction < FLCE_REDUCTION_NONE || p->reduction > FLCE_REDUCTION_MEAN) return FLCE_ERR_INVALID_ARG;
  if ((p->flags & ~FLCE_OFFSETS_INT32) != 0 || p->length_normalize < 0 || p->length_normalize > 1 ||
      p->reserved != 0)
    return FLCE_ERR_INVALID_ARG;
  if (!isfinite(p->beta) || !(p->beta > 0.0) || !isfinite(p->margin)) return FLCE_ERR_INVALID_ARG;
  if (!(p->label_smoothing >= 0.0 && p->label_smoothing <= 1.0)) return FLCE_ERR_INVALID_ARG;
  if (p->label_smoothing != 0.0 && p->type != FLCE_PREFERENCE_SIGMOID) return FLCE_ERR_INVALID_ARG;
  return FLCE_OK;
}

static int check_policy(const flce_policy_params* p) {
  if (!p || p->n_seqs < 0 || p->length < 0 || !align_dtype_ok(p->dtype)) return FLCE_ERR_INVALID_ARG;
  if (p->reduction < FLCE_REDUCTION_NONE || p->reduction > FLCE_REDUCTION_SEQUENCE_MEAN) return FLCE_ERR_INVALID_ARG;
  if ((p->flags & ~(FLCE_OFFSETS_INT32 | FLCE_ADVANTAGE_PER_SEQUENCE)) != 0 || p->reserved != 0)
    return FLCE_ERR_INVALID_ARG;
  if (!(p->clip_low >= 0.0) || !(p->clip_high >= 0.0)) return FLCE_ERR_INVALID_ARG;
  if (!(p->dual_clip == 0.0 || (p->dual_clip > 1.0 && isfinite(p->dual_clip)))) return FLCE_ERR_INVALID_ARG;
  if (!isfinite(p->kl_coef) || !isfinite(p->entropy_coef)) return FLCE_ERR_INVALID_ARG;
  return FLCE_OK;
}

}  // namespace flce

using namespace flce;

extern "C" {

int flce_preference_workspace_size(const flce_preference_params* p, size_t* bytes) {
  if (!bytes) return FLCE_ERR_INVALID_ARG;
  int rc = check_preference(p);
  if (rc != FLCE_OK) return rc;
  const int64_t n = max_slots(p->n_seqs, p->length, &rc);
  if (rc != FLCE_OK) return rc;
  *bytes = align256(size_t(n > 0 ? n : 1) * sizeof(SeqPart));
  return FLCE_OK;
}

int flce_preference_forward(const flce_preference_params* p, flce_token_view logps, flce_token_view ref_logps,
                            flce_token_view mask, const void* offsets, float* loss, float* rewards, float* seq_grad,
                            void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int rc = flce_preference_workspace_size(p, &need);
  if (rc != FLCE_OK) return rc;
  PreferenceArgs a;
  memset(&a, 0, sizeof(a));
  rc = plan_seqs(p->n_seqs, p->length, offsets != nullptr, &a.q);
  if (rc != FLCE_OK) return rc;
  const bool tokens = a.q.waves > 0;
  if (!workspace || (tokens && !logps.data)) return FLCE_ERR_INVALID_ARG;
  if (!loss && (p->reduction != FLCE_REDUCTION_NONE || p->n_seqs > 0)) return FLCE_ERR_INVALID_ARG;
  if (p->n_seqs > 0 && (!rewards || !seq_grad)) return FLCE_ERR_INVALID_ARG;
  bool vec = true;
  const size_t e = esize_of(p->dtype);
  if ((rc = check_layout(mask, offsets, p->flags, &a.q, &vec)) != FLCE_OK) return rc;
  if ((rc = check_view(logps, a.q, e, &a.ld_logps, &vec)) != FLCE_OK) return rc;
  if ((rc = check_view(ref_logps, a.q, e, &a.ld_ref, &vec)) != FLCE_OK) return rc;
  if (!aligned(loss, 4) || !aligned(rewards, 4) || !aligned(seq_grad, 4) || !aligned(workspace, 16))
    return FLCE_ERR_UNSUPPORTED;
  if (workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  a.logps = logps.data;
  a.ref = ref_logps.data;
  a.slots = static_cast<SeqPart*>(workspace);
  a.loss = loss;
  a.rewards = rewards;
  a.seq_grad = seq_grad;
  a.reduction = p->reduction;
  a.type = p->type;
  a.normalize = p->length_normalize;
  a.group = slot_group(a.q);
  a.beta = p->beta;
  a.smoothing = p->label_smoothing;
  a.margin = p->margin;
  return launch_preference(p->dtype, vec, a, static_cast<hipStream_t>(stream)) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

int flce_preference_backward(const flce_preference_params* p, const float* grad_loss, const float* seq_grad,
                             flce_token_view mask, const void* offsets, void* grad_logps, void* stream) {
  int rc = check_preference(p);
  if (rc != FLCE_OK) return rc;
  PreferenceGradArgs a;
  memset(&a, 0, sizeof(a));
  rc = plan_seqs(p->n_seqs, p->length, offsets != nullptr, &a.q);
  if (rc != FLCE_OK) return rc;
  if (a.q.waves > 0 && !grad_logps) return FLCE_ERR_INVALID_ARG;
  // (a packed buffer may hold no sequence at all: its gradient is 0)
  if (p->n_seqs > 0 && !seq_grad) return FLCE_ERR_INVALID_ARG;
  if (!grad_loss && (p->reduction != FLCE_REDUCTION_NONE || p->n_seqs > 0)) return FLCE_ERR_INVALID_ARG;
  bool vec = true;
  if ((rc = check_layout(mask, offsets, p->flags, &a.q, &vec)) != FLCE_OK) return rc;
  const size_t e = esize_of(p->dtype);
  if (!aligned(grad_loss, 4) || !aligned(seq_grad, 4) || !aligned(grad_logps, e)) return FLCE_ERR_UNSUPPORTED;
  if (!aligned(grad_logps, 4 * e)) vec = false;
  a.grad_loss = grad_loss;
  a.seq_grad = seq_grad;
  a.per_pair = p->reduction == FLCE_REDUCTION_NONE;
  a.grad_logps = grad_logps;
  return launch_preference_grad(p->dtype, vec, a, static_cast<hipStream_t>(stream)) == hipSuccess ? FLCE_OK
                                                                                                  : FLCE_ERR_HIP;
}

int flce_policy_workspace_size(const flce_policy_params* p, size_t* bytes) {
  if (!bytes) return FLCE_ERR_INVALID_ARG;
  int rc = check_policy(p);
  if (rc != FLCE_OK) return rc;
  const int64_t n = max_slots(p->n_seqs, p->length, &rc);
  if (rc != FLCE_OK) return rc;
  *bytes = align256(size_t(n > 0 ? n : 1) * (sizeof(SeqPart) + sizeof(WavePart)));
  return FLCE_OK;
}

int flce_policy_forward(const flce_policy_params* p, flce_token_view logps, flce_token_view old_logps,
                        flce_token_view ref_logps, flce_token_view entropy, flce_token_view advantages,
                        flce_token_view mask, const void* offsets, float* loss, float* unit_grad, float* weights,
                        flce_policy_metrics* metrics, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int rc = flce_policy_workspace_size(p, &need);
  if (rc != FLCE_OK) return rc;
  PolicyArgs a;
  memset(&a, 0, sizeof(a));
  rc = plan_seqs(p->n_seqs, p->length, offsets != nullptr, &a.q);
  if (rc != FLCE_OK) return rc;
  const bool tokens = a.q.waves > 0;
  const bool per_seq = (p->flags & FLCE_ADVANTAGE_PER_SEQUENCE) != 0;
  if (!workspace || !weights) return FLCE_ERR_INVALID_ARG;
  if (tokens && (!logps.data || !old_logps.data)) return FLCE_ERR_INVALID_ARG;
  if ((per_seq ? p->n_seqs > 0 : tokens) && !advantages.data) return FLCE_ERR_INVALID_ARG;
  if (!loss && (p->reduction != FLCE_REDUCTION_NONE || tokens)) return FLCE_ERR_INVALID_ARG;
  if (p->kl_coef != 0.0 && tokens && !ref_logps.data) return FLCE_ERR_INVALID_ARG;
  if (p->entropy_coef != 0.0 && tokens && !entropy.data) return FLCE_ERR_INVALID_ARG;
  bool vec = true;
  const size_t e = esize_of(p->dtype);
  if ((rc = check_layout(mask, offsets, p->flags, &a.q, &vec)) != FLCE_OK) return rc;
  if ((rc = check_view(logps, a.q, e, &a.ld_logps, &vec)) != FLCE_OK) return rc;
  if ((rc = check_view(old_logps, a.q, e, &a.ld_old, &vec)) != FLCE_OK) return rc;
  if ((rc = check_view(ref_logps, a.q, e, &a.ld_ref, &vec)) != FLCE_OK) return rc;
  if ((rc = check_view(entropy, a.q, e, &a.ld_entropy, &vec)) != FLCE_OK) return rc;
  if (per_seq) {
    if (!aligned(advantages.data, 4)) return FLCE_ERR_UNSUPPORTED;
  } else if ((rc = check_view(advantages, a.q, 4, &a.ld_adv, &vec)) != FLCE_OK) {
    return rc;
  }
  if (!aligned(loss, 4) || !aligned(unit_grad, 16) || !aligned(weights, 4) || !aligned(metrics, 8) ||
      !aligned(workspace, 16))
    return FLCE_ERR_UNSUPPORTED;
  if (p->reduction == FLCE_REDUCTION_NONE && !aligned(loss, 16)) vec = false;
  if (workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  a.logps = logps.data;
  a.old = old_logps.data;
  a.ref = ref_logps.data;
  a.entropy = entropy.data;
  a.adv = static_cast<const float*>(advantages.data);
  a.adv_per_seq = per_seq;
  a.reduction = p->reduction;
  a.group = slot_group(a.q);
  const double low = 1.0 - p->clip_low, high = 1.0 + p->clip_high;
  a.low = (float)low;
  a.high = (float)high;
  a.dual = (float)p->dual_clip;
  a.log_low = low > 0.0 ? log(low) : -INFINITY;
  a.log_high = log(high);
  a.log_dual = p->dual_clip > 0.0 ? log(p->dual_clip) : INFINITY;
  a.kl_coef = (float)p->kl_coef;
  a.entropy_coef = (float)p->entropy_coef;
  const int64_t slots = slot_count(a.q);
  a.slots = static_cast<SeqPart*>(workspace);
  a.parts = reinterpret_cast<WavePart*>(a.slots + slots);
  a.loss = loss;
  a.unit_grad = unit_grad;
  a.weights = weights;
  a.metrics = metrics;
  return launch_policy(p->dtype, vec, a, static_cast<hipStream_t>(stream)) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

int flce_policy_backward(const flce_policy_params* p, const float* grad_loss, const float* unit_grad,
                         const float* weights, flce_token_view mask, const void* offsets, void* grad_logps,
                         void* grad_entropy, void* stream) {
  int rc = check_policy(p);
  if (rc != FLCE_OK) return rc;
  PolicyGradArgs a;
  memset(&a, 0, sizeof(a));
  rc = plan_seqs(p->n_seqs, p->length, offsets != nullptr, &a.q);
  if (rc != FLCE_OK) return rc;
  const bool tokens = a.q.waves > 0;
  if (!weights || (tokens && grad_logps && !unit_grad)) return FLCE_ERR_INVALID_ARG;
  if (!grad_loss && (p->reduction != FLCE_REDUCTION_NONE || tokens)) return FLCE_ERR_INVALID_ARG;
  bool vec = true;
  if ((rc = check_layout(mask, offsets, p->flags, &a.q, &vec)) != FLCE_OK) return rc;
  const size_t e = esize_of(p->dtype);
  if (!aligned(grad_loss, 4) || !aligned(unit_grad, 16) || !aligned(weights, 4) || !aligned(grad_logps, e) ||
      !aligned(grad_entropy, e))
    return FLCE_ERR_UNSUPPORTED;
  if (!aligned(grad_logps, 4 * e) || !aligned(grad_entropy, 4 * e)) vec = false;
  a.per_token = p->reduction == FLCE_REDUCTION_NONE;
  if (a.per_token && !aligned(grad_loss, 16)) vec = false;
  a.grad_loss = grad_loss;
  a.unit_grad = unit_grad;
  a.weights = weights;
  a.seq_weights = p->reduction == FLCE_REDUCTION_SEQUENCE_MEAN;
  a.entropy_coef = (float)p->entropy_coef;
  a.grad_logps = grad_logps;
  a.grad_entropy = grad_entropy;
  if (!grad_logps && !grad_entropy) return FLCE_OK;
  return launch_policy_grad(p->dtype, vec, a, static_cast<hipStream_t>(stream)) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

}  // extern "C"
