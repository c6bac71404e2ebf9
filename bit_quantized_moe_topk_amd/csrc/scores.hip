// Routing by scores: sigmoid or softmax scores, a bias that takes part in the
// selection alone, groups of experts, top-k and gates, and the gates' gradient
// for the logits.
//
// One wave a token. What is ranked (score + bias) is held in 64 bits: in 32,
// two experts a last place apart would come in the order of their roundings.
#include "gemv.h"
#include "norm.h"
#include "topk.h"

namespace moe {
namespace {

// Order-preserving code of a double: NaN is 1, below -inf; 0 marks what cannot be selected.
__device__ inline uint64_t orderable64(double v) {
  if (v != v) return 1ull;
  const uint64_t u = __double_as_longlong(v == 0.0 ? 0.0 : v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
constexpr uint64_t kOff = 0x000FFFFFFFFFFFFFull;  // -inf's code
__device__ inline double from_orderable64(uint64_t o) {
  return __longlong_as_double((o >> 63) ? (o & 0x7FFFFFFFFFFFFFFFull) : ~o);
}

__device__ inline double wave_max64(double v) {
  for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ inline double wave_sum64(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

__device__ inline float logit_at(const ScoreArgs& a, int t, int e) {
  const size_t at = (size_t)t * a.ld + e;
  return a.bf16 ? bf16_lo(static_cast<const uint16_t*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
}

constexpr int kWaves = 4;  // tokens per workgroup

template <int P>
__global__ __launch_bounds__(64 * kWaves) void scores_forward(ScoreArgs a) {
  __shared__ double values[kWaves][64 * P];
  __shared__ uint64_t keys[kWaves][64 * P];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  double s[P];
  uint64_t key[P];
  float l[P];
#pragma unroll
  for (int i = 0; i < P; ++i) l[i] = logit_at(a, t, min(lane + 64 * i, a.E - 1));
  double top = -INFINITY, total = 0.0;
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < P; ++i) top = fmax(top, (double)l[i]);
    top = wave_max64(top);
    bool nan = false;  // (a maximum leaves it out)
#pragma unroll
    for (int i = 0; i < P; ++i) nan |= l[i] != l[i];
    if (__any(nan)) top = NAN;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 64 * i < a.E) total += top == -INFINITY ? 0.0 : exp((double)l[i] - top);
    total = wave_sum64(total);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    s[i] = !a.softmax ? 1.0 / (1.0 + exp(-(double)l[i])) : top == -INFINITY ? 0.0 : exp((double)l[i] - top) / total;
    double c = !a.bias ? (double)l[i] : s[i] + (double)a.bias[min(e, a.E - 1)];
    if (l[i] == -INFINITY) c = -INFINITY;
    key[i] = e < a.E ? orderable64(c) : 0ull;
    values[wave][e] = s[i];
    keys[wave][e] = key[i];
  }
  __builtin_amdgcn_wave_barrier();
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    uint64_t mine = 0;
    if (lane < a.groups) {
      uint64_t k1 = kOff, k2 = kOff;  // what is not above -inf is left out
      int e1 = 0, e2 = 0;
      for (int e = lane * size; e < (lane + 1) * size; ++e) {
        const uint64_t k = keys[wave][e];
        if (k > k1) {
          k2 = k1;
          e2 = e1;
          k1 = k;
          e1 = e;
        } else if (k > k2) {
          k2 = k;
          e2 = e;
        }
      }
      mine = k1;
      if (a.group_top == 2 && k1 > kOff) {
        const double v1 = a.bias ? from_orderable64(k1) : values[wave][e1];
        const double v2 = k2 == kOff ? 0.0 : a.bias ? from_orderable64(k2) : values[wave][e2];
        mine = orderable64(v1 + v2);
      }
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t o = __shfl(mine, g, 64);
      rank += o > mine || (o == mine && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.keep);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 64 * i < a.E && !(kept >> ((lane + 64 * i) / size) & 1)) key[i] = 0ull;
  }
  double sum = 0.0;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = key[0];
    int e = lane;
#pragma unroll
    for (int i = 1; i < P; ++i)
      if (key[i] > best) {
        best = key[i];
        e = lane + 64 * i;
      }
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t ob = __shfl_xor(best, o, 64);
      const int oe = __shfl_xor(e, o, 64);
      if (ob > best || (ob == best && oe < e)) {
        best = ob;
        e = oe;
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 64 * i == e) key[i] = 0ull;
    if (lane == 0) a.idx[(size_t)t * a.k + j] = e;
    sum += values[wave][e];
  }
  __threadfence_block();
  for (int j = lane; j < a.k; j += 64) {
    const double v = values[wave][a.idx[(size_t)t * a.k + j]];
    a.gates[(size_t)t * a.k + j] = (float)((double)a.scale * (!a.renorm ? v : sum == 0.0 ? 0.0 : v / sum));
  }
}

template <int P>
__global__ __launch_bounds__(64 * kWaves) void scores_backward(ScoreArgs a) {
  __shared__ float row[kWaves][64 * P];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  const int32_t* idx = a.idx + (size_t)t * a.k;
  const float* dg = a.d_gates + (size_t)t * a.k;
#pragma unroll
  for (int i = 0; i < P; ++i) row[wave][lane + 64 * i] = 0.f;
  // the scores' base: over the row, or with renorm over what was selected
  float top = -INFINITY, total = 0.f, l[P];
  bool nan = false;  // (a maximum leaves it out)
  if (a.softmax && !a.renorm) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      l[i] = lane + 64 * i < a.E ? logit_at(a, t, lane + 64 * i) : -INFINITY;
      top = fmaxf(top, l[i]);
      nan |= l[i] != l[i];
    }
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if (__any(nan)) top = NAN;
#pragma unroll
    for (int i = 0; i < P; ++i) total += top == -INFINITY ? 0.f : expf(l[i] - top);
    total = wave_sum(total);
  } else if (a.softmax) {
    for (int j = lane; j < a.k; j += 64)
      if ((unsigned)idx[j] < (unsigned)a.E) {
        const float v = logit_at(a, t, idx[j]);
        top = fmaxf(top, v);
        nan |= v != v;
      }
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if (__any(nan)) top = NAN;
    total = 1.f;
  }
  auto score = [&](float v) {
    return !a.softmax ? 1.f / (1.f + expf(-v)) : top == -INFINITY ? 0.f : expf(v - top) / total;
  };
  float S = 0.f, D = 0.f;  // sums of the selected scores and of d times them
  for (int j = lane; j < a.k; j += 64)
    if ((unsigned)idx[j] < (unsigned)a.E) {
      const float s = score(logit_at(a, t, idx[j]));
      S += s;
      D = fmaf(a.scale * dg[j], s, D);
    }
  S = wave_sum(S);
  D = wave_sum(D);
  const float mean = a.renorm ? (S == 0.f ? 0.f : D / S) : 0.f, inv = a.renorm ? (S == 0.f ? 0.f : 1.f / S) : 1.f;
  __builtin_amdgcn_wave_barrier();
  for (int j = 0; j < a.k; ++j) {  // (in order: an index may come twice)
    const int e = idx[j];
    if ((unsigned)e < (unsigned)a.E && lane == 0) row[wave][e] += (a.scale * dg[j] - mean) * inv;
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    if (e >= a.E) continue;
    const float d = row[wave][e];
    float v = 0.f;
    if (a.softmax && !a.renorm) {
      v = score(l[i]) * (d - D);
    } else if (d != 0.f) {
      const float s = score(logit_at(a, t, e));
      v = a.softmax ? s * d : d * s * (1.f - s);
    }
    const size_t at = (size_t)t * a.E + e;
    if (a.bf16) static_cast<uint16_t*>(a.dlogits)[at] = (uint16_t)f32_to_bf16_bits(v);
    else static_cast<float*>(a.dlogits)[at] = v;
  }
}

}  // namespace

#define BY_LANES(M) \
  const int per = (a.E + 63) / 64; \
  if (per <= 1) { M(1); } \
  else if (per <= 2) { M(2); } \
  else if (per <= 4) { M(4); } \
  else if (per <= 8) { M(8); } \
  else if (per <= 16) { M(16); } \
  else { M(32); }

hipError_t launch_scores(const ScoreArgs& a, hipStream_t s) {
  const dim3 g((a.T + kWaves - 1) / kWaves);
#define FORWARD(P) MOE_LAUNCH("scores", s, scores_forward<P>, g, dim3(64 * kWaves), 0, s, a)
  BY_LANES(FORWARD)
#undef FORWARD
  return hipGetLastError();
}

hipError_t launch_scores_backward(const ScoreArgs& a, hipStream_t s) {
  const dim3 g((a.T + kWaves - 1) / kWaves);
#define BACKWARD(P) MOE_LAUNCH("scores_backward", s, scores_backward<P>, g, dim3(64 * kWaves), 0, s, a)
  BY_LANES(BACKWARD)
#undef BACKWARD
  return hipGetLastError();
}

}  // namespace moe
