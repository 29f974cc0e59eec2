// Token embedding: kernel arguments, plan and launchers (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/flce.h"

namespace flce {

constexpr int kSortAlone = 16384;    // tokens up to which the sort is one launch
constexpr int kSortBits = 9;         // of a pass: two for a vocabulary below 2^18
constexpr int kSortBins = 1 << kSortBits;

struct EmbedPlan {
  int64_t n, v;
  int h;
  int dtype, grad_dtype;
  bool ids_i32, accumulate;
  float scale;
  int64_t ignore_index;
  // backward
  int passes;                  // of the sort, kSortBits each
  int sort_parts;              // one launch: workgroups, each with the ids of its part
  int sort_waves, sort_blocks; // else: waves of a workgroup (512 ids each), workgroups
  int chunk;                   // sorted ids a workgroup sums
  int64_t n_chunks;
  size_t w_keys[2], w_at[2], w_hist, w_part, w_bytes;   // workspace offsets
};

void plan_embedding_backward(EmbedPlan* p);
hipError_t launch_embedding_forward(const EmbedPlan& p, const void* ids, const void* weight, void* out, hipStream_t st);
hipError_t launch_embedding_backward(const EmbedPlan& p, const void* ids, const void* grad, void* grad_weight, char* ws,
                                     hipStream_t st);

}  // namespace flce
