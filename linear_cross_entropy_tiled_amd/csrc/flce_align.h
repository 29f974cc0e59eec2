// Preference and policy losses: kernel arguments and launchers (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/flce.h"

namespace flce {

// S sequences of tokens, padded or packed, and how waves share them.
struct Seqs {
  int64_t S, length;           // packed: length = tokens in all
  int64_t chunk;               // tokens per wave, a multiple of 256
  int64_t chunks_per_row;      // padded
  int64_t waves;
  const void* offsets;
  const uint8_t* mask;         // NULL: every token counts
  int64_t ld_mask;
  int packed, off_i32;
};

// A wave's partial sum of one sequence.
struct SeqPart {
  double sum;
  int count, pad;
};

struct PreferenceArgs {
  Seqs q;
  const void* logps;
  const void* ref;
  int64_t ld_logps, ld_ref;
  SeqPart* slots;
  float* loss;
  float* rewards;
  float* seq_grad;
  int reduction, type, normalize;
  int group;                   // lanes that add one sequence's slots
  double beta, smoothing, margin;
};

struct PreferenceGradArgs {
  Seqs q;
  const float* grad_loss;
  const float* seq_grad;
  int per_pair;
  void* grad_logps;
};

// A wave's share of the policy loss's metrics.
struct WavePart {
  double kl;
  int clipped, kept;
};

struct PolicyArgs {
  Seqs q;
  const void* logps;
  const void* old;
  const void* ref;
  const void* entropy;
  const float* adv;
  int64_t ld_logps, ld_old, ld_ref, ld_entropy, ld_adv;
  int adv_per_seq, reduction, group;
  float low, high, dual;       // clipping borders of the ratio; dual 0 = off
  double log_low, log_high, log_dual;
  float kl_coef, entropy_coef;
  SeqPart* slots;
  WavePart* parts;
  float* loss;
  float* unit_grad;
  float* weights;
  flce_policy_metrics* metrics;
};

struct PolicyGradArgs {
  Seqs q;
  const float* grad_loss;
  const float* unit_grad;
  const float* weights;
  int per_token, seq_weights;
  float entropy_coef;
  void* grad_logps;
  void* grad_entropy;
};

hipError_t launch_preference(int dtype, bool vec, const PreferenceArgs& a, hipStream_t st);
hipError_t launch_preference_grad(int dtype, bool vec, const PreferenceGradArgs& a, hipStream_t st);
hipError_t launch_policy(int dtype, bool vec, const PolicyArgs& a, hipStream_t st);
hipError_t launch_policy_grad(int dtype, bool vec, const PolicyGradArgs& a, hipStream_t st);

}  // namespace flce
