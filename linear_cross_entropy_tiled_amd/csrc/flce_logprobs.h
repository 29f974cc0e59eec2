// Log-probabilities of a linear head: plan, kernel arguments and launchers (internal).
#pragma once

#include "flce_internal.h"

namespace flce {

// How a log-probability call runs: which kernels, and its workspace (offsets; the
// backward's regions follow the loss backward's, b_*).
struct LpPlan {
  // forward: the first vt_large vocabulary tiles run as 256 x 256 tiles in S_large
  // splits, the rest of the vocabulary as 64 x bn tiles in S_small splits
  int bn;
  int vt_large, S_large, S_small;
  int N_pad;
  // MXFP4: hidden states' codes and scales where they are quantised in the call; scale rows
  // of a length that is no multiple of 4 are copied to rows of ld_mx
  int ld_mx;
  size_t f_q, f_hmx, f_wmx;
  size_t f_tmx_w, f_tmx_h;    // scales in the large tiles' order
  size_t f_bytes;

  // Up to 64 tokens in 16 bits: the logit gradient is held as the sum of two 16-bit
  // rows per token, its rounding and the rest.  One rounding of each entry, relative to
  // the output's own, averages out over many tokens (the gradients' error against fp64
  // is 1.4 times that of rounding the outputs alone); of few tokens' gradients one entry
  // can be most (2.5 times).  Costs a second row in two contractions that are bound by
  // reading or writing the weight there.
  bool split;
  bool d_small, gw_small, gh_small;
  int n64, N64;           // 64-token tiles, padded tokens
  int K_pad;              // tokens the grad_weight contraction runs over
  int gh_parts, gh_kt;    // grad_hidden: splits over the vocabulary (128-byte stages each)
  size_t b_coefE, b_gbpart, b_ghpart, b_bytes;
};

// Upstream gradients of flce_logprobs_backward; NULL = zero.
struct LpGrad {
  const float* grad_logps;
  const float* grad_entropy;
  const float* entropy;   // the forward's (with grad_entropy)
};

struct LpTileArgs {
  const char* hidden;
  const char* weight;
  const void* bias;           // the operands' type; fp32 for int8
  const float* hidden_scale;  // int8
  const float* weight_scale;  // int8
  const uint8_t* hidden_mx;   // MXFP4: scale bytes, rows of ld_hmx (a multiple of 4)
  const uint8_t* weight_mx;
  uint32_t ld_hmx, ld_wmx;
  const uint8_t* hidden_tmx;  // the same in the large tiles' order (launch_mx_prep)
  const uint8_t* weight_tmx;
  const void* targets;
  int tgt_i32;
  int N, H, V;                // H: elements of a row, of MXFP4 its bytes
  int64_t ignore_index;
  float scale, cap;
  int v_first;                // first vocabulary row of the launch
  int n_vt, S;                // its vocabulary tiles (256 or 64 rows) and splits
  int S_all, s_first, N_pad;
  float* part;                // [4][S_all][N_pad]: m, l, T, y_t; this launch's splits from s_first on
  int* status;                // set to FLCE_OK here; lp_rows_kernel reports bad targets
};

void plan_logprobs(const Plan& pl, LpPlan* lp);
// pl.int8, pl.mx: 8- and 4-bit operands with their scales (fp32 and bytes), bias in fp32; of pl.mx hidden may be values
// of pl.x_dtype, without scales.
hipError_t launch_logprobs(const Plan& pl, const LpPlan& lp, const void* hidden, const void* weight, const void* bias,
                           const void* hidden_scale, const void* weight_scale, const void* targets, float* logps,
                           float* entropy, float* lse, char* ws, hipStream_t st);
hipError_t launch_logprobs_backward(const Plan& pl, const LpPlan& lp, const LpGrad& g, const void* hidden,
                                    const void* weight, const void* bias, const void* targets, const float* lse,
                                    void* grad_hidden, void* grad_weight, void* grad_bias, char* ws, hipStream_t st);
hipError_t launch_quantize(int dtype, const void* x, int64_t rows, int64_t cols, int8_t* q, float* scale,
                           hipStream_t st);

// MXFP4's large tiles (flce_mx_tiles.hip): nwg workgroups, token tile by split.
void launch_mx_tiles(const Plan& pl, const LpTileArgs& a, int nwg, hipStream_t st);

// Small-tile kernels (flce_small.hip).
void launch_lp_small(const Plan& pl, int bn, const LpTileArgs& a, int n_tt, hipStream_t st);
void launch_dlogits_small(const Plan& pl, const DlogitsArgs& d, hipStream_t st);
void launch_gw_small(int dtype, const GwArgs& g, hipStream_t st);
void launch_gh_small(int dtype, const GhArgs& h, hipStream_t st);

}  // namespace flce
