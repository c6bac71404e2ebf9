// Internal declarations of the RMS norm (norm.hip) and of routing by scores (scores.hip).
#pragma once

#include "common.h"

namespace moe {

size_t norm_workspace_bytes(int T, int H);
hipError_t launch_norm(const void* x, int dtype, long long ldx, const void* residual, long long ldr, const void* weight,
                       int wdtype, float eps, int T, int H, void* total, void* y, uint8_t* codes, float* scales,
                       hipStream_t s);
hipError_t launch_norm_backward(const void* dy, long long ldd, const void* h, long long ldh, int dtype, const void* weight,
                                int wdtype, const void* d_total, long long ldt, float eps, int T, int H, void* dh,
                                float* dweight, void* ws, hipStream_t s);

struct ScoreArgs {
  const void* logits;
  long long ld;
  int bf16, T, E, k;
  const float* bias;
  int softmax, groups, keep, group_top, renorm;
  float scale;
  int32_t* idx;
  float* gates;
  const float* d_gates;
  void* dlogits;
};
hipError_t launch_scores(const ScoreArgs& a, hipStream_t s);
hipError_t launch_scores_backward(const ScoreArgs& a, hipStream_t s);

}  // namespace moe
