// Per-expert counts, balance loss and z loss of a router, and their gradient
// for the logits.
//
// Over the n tokens that the mask keeps, with p the softmax of a token's
// logits and lse its log-sum-exp:
//   counts[e] = kept assignments to e,  f_e = counts[e] / (n k)
//   balance   = E sum_e f_e mean_t p_te = E / n sum_t (f . p_t)
//   z         = mean_t lse_t^2
//   d logit_te = p_te (g_b E / n (f_e - f . p_t) + g_z 2 lse_t / n)
// f depends on idx alone. So the counts are taken first, and then one pass over
// the logits, one wave a token, gives both losses through the two scalars
// f . p_t and lse_t: no column sums of p, and nothing as large as the logits,
// is kept. The gradient is one more pass that reads the logits and writes as
// many values. Bound by those bytes; small batches by their launches.
//
// Sums are float32 in a fixed order (per wave over its tokens, then over the
// waves in order), counts are integers: results do not vary from run to run.
#include "common.h"
#include "gemv.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int kWaves = 4;         // tokens in flight per workgroup
constexpr int kCountIds = 4096;   // ids per counting workgroup
constexpr int kCountGroups = 64;  // most counting workgroups
constexpr int kRowGroups = 512;   // most workgroups of the pass over the logits

struct BalanceArgs {
  const void* logits;
  long long ld;
  int bf16, T, E, k;
  const int32_t* idx;
  const uint8_t* keep;  // [T] or null
  int32_t* counts;      // [E]
  int32_t* kept;        // [1]
  float* losses;        // [2]
  const float* d;       // [2]
  void* dx;             // [T][E]
  int32_t* wcounts;     // workspace: [G][E + 1] counts of each counting workgroup, its kept tokens last
  float* wsums;         // [kRowGroups][2]
  uint32_t* done;
};

__device__ inline float load_logit(const BalanceArgs& a, size_t i) {
  return a.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[i] << 16)
                : static_cast<const float*>(a.logits)[i];
}

// Counting workgroup b of G: the ids of tokens [b T / G, (b + 1) T / G) in an LDS histogram.
__global__ __launch_bounds__(256) void balance_count(BalanceArgs a) {
  __shared__ int32_t h[MOE_MAX_E_DEV + 1];
  const int G = gridDim.x, b = blockIdx.x, tid = threadIdx.x;
  for (int e = tid; e <= a.E; e += 256) h[e] = 0;
  __syncthreads();
  const int t0 = (int)((long long)b * a.T / G), t1 = (int)((long long)(b + 1) * a.T / G);
  for (long long i = (long long)t0 * a.k + tid; i < (long long)t1 * a.k; i += 256) {
    const int e = a.idx[i];
    if ((unsigned)e < (unsigned)a.E && (!a.keep || a.keep[i / a.k])) atomicAdd(&h[e], 1);
  }
  int n = 0;
  for (int t = t0 + tid; t < t1; t += 256) n += !a.keep || a.keep[t] ? 1 : 0;
  if (n) atomicAdd(&h[a.E], n);
  __syncthreads();
  for (int e = tid; e <= a.E; e += 256) a.wcounts[(size_t)b * (a.E + 1) + e] = h[e];
  if (b == 0 && tid == 0) *a.done = 0u;
}

// A token's logits in registers (column lane + 64 i in slot i), exp(x - max)
// in their place; *lse and 1 / sum. A token whose logits are all -inf has no
// distribution: p is 0 and lse 0.
template <int P>
__device__ inline void softmax_row(const BalanceArgs& a, int t, float (&x)[P], float* lse, float* inv) {
  const int lane = threadIdx.x & 63;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    x[i] = lane + 64 * i < a.E ? load_logit(a, (size_t)t * a.ld + lane + 64 * i) : -INFINITY;
    top = fmaxf(top, x[i]);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  float sum = 0.f;
  const bool none = top == -INFINITY;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    // NaN logits pass fmaxf by, and come back in here
    x[i] = none && x[i] == -INFINITY ? 0.f : expf(x[i] - top);
    sum += x[i];
  }
  sum = wave_sum(sum);
  *inv = sum == 0.f ? 0.f : 1.f / sum;
  *lse = sum == 0.f ? 0.f : top + logf(sum);
}

// f[slot] / (n k) of this lane's columns, from the finished counts.
template <int P>
__device__ inline void load_share(const int32_t* counts, int n, const BalanceArgs& a, float (&f)[P]) {
  const int lane = threadIdx.x & 63;
  const float total = (float)n * (float)a.k;
#pragma unroll
  for (int i = 0; i < P; ++i)
    f[i] = lane + 64 * i < a.E && n > 0 ? (float)counts[lane + 64 * i] / total : 0.f;
}

// Pass over the logits. Every workgroup adds up the counting workgroups'
// counts (the first also writes them out); the last one to finish adds up the
// workgroups' sums in order.
template <int P>
__global__ __launch_bounds__(64 * kWaves) void balance_rows(BalanceArgs a, int G) {
  __shared__ int32_t cnt[MOE_MAX_E_DEV + 1];
  __shared__ float ws[kWaves][2];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= a.E; e += 64 * kWaves) {
    int c = 0;
    for (int b = 0; b < G; ++b) c += a.wcounts[(size_t)b * (a.E + 1) + e];
    cnt[e] = c;
    if (blockIdx.x == 0) {
      if (e < a.E) a.counts[e] = c;
      else *a.kept = c;
    }
  }
  __syncthreads();
  const int n = cnt[a.E];
  float f[P], fp = 0.f, zz = 0.f;
  load_share<P>(cnt, n, a, f);
  for (int t = blockIdx.x * kWaves + wave; t < a.T; t += gridDim.x * kWaves) {
    if (a.keep && !a.keep[t]) continue;
    float x[P], lse, inv, dot = 0.f;
    softmax_row<P>(a, t, x, &lse, &inv);
#pragma unroll
    for (int i = 0; i < P; ++i) dot = fmaf(f[i], x[i], dot);
    fp += wave_sum(dot) * inv;
    zz += lse * lse;
  }
  if (lane == 0) {
    ws[wave][0] = fp;
    ws[wave][1] = zz;
  }
  __syncthreads();
  if (tid == 0) {
    float s0 = 0.f, s1 = 0.f;
    for (int w = 0; w < kWaves; ++w) {
      s0 += ws[w][0];
      s1 += ws[w][1];
    }
    __hip_atomic_store(&a.wsums[2 * blockIdx.x], s0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&a.wsums[2 * blockIdx.x + 1], s1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last || wave) return;
  float s0 = 0.f, s1 = 0.f;
  for (int b = lane; b < (int)gridDim.x; b += 64) {
    s0 += __hip_atomic_load(&a.wsums[2 * b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s1 += __hip_atomic_load(&a.wsums[2 * b + 1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  s0 = wave_sum(s0);
  s1 = wave_sum(s1);
  if (lane == 0) {
    a.losses[0] = n ? s0 * ((float)a.E / (float)n) : 0.f;
    a.losses[1] = n ? s1 / (float)n : 0.f;
  }
}

template <int P>
__global__ __launch_bounds__(64 * kWaves) void balance_gradient(BalanceArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = *a.kept;
  float f[P];
  load_share<P>(a.counts, n, a, f);
  const float cb = n ? a.d[0] * ((float)a.E / (float)n) : 0.f, cz = n ? a.d[1] * (2.f / (float)n) : 0.f;
  for (int t = blockIdx.x * kWaves + wave; t < a.T; t += gridDim.x * kWaves) {
    float x[P], lse = 0.f, inv = 0.f, dot = 0.f;
    const bool keep = !a.keep || a.keep[t];
    if (keep) {
      softmax_row<P>(a, t, x, &lse, &inv);
#pragma unroll
      for (int i = 0; i < P; ++i) dot = fmaf(f[i], x[i], dot);
      dot = wave_sum(dot) * inv;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane + 64 * i;
      if (e >= a.E) continue;
      const float v = keep ? x[i] * inv * fmaf(cb, f[i] - dot, cz * lse) : 0.f;
      if (a.bf16) static_cast<uint16_t*>(a.dx)[(size_t)t * a.E + e] = (uint16_t)f32_to_bf16_bits(v);
      else static_cast<float*>(a.dx)[(size_t)t * a.E + e] = v;
    }
  }
}

int count_groups(int T, int k) {
  const long long g = ((long long)T * k + kCountIds - 1) / kCountIds;
  return (int)(g < 1 ? 1 : g > kCountGroups ? kCountGroups : g);
}

int row_groups(int T) {
  const int g = (T + kWaves - 1) / kWaves;
  return g < 1 ? 1 : g > kRowGroups ? kRowGroups : g;
}

template <int P>
void launch_rows(const BalanceArgs& a, hipStream_t s) {
  MOE_LAUNCH("balance_rows", s, balance_rows<P>, dim3(row_groups(a.T)), dim3(64 * kWaves), 0, s, a,
             count_groups(a.T, a.k));
}
template <int P>
void launch_grad(const BalanceArgs& a, hipStream_t s) {
  const int g = (a.T + kWaves - 1) / kWaves, most = 8 * device_cus();
  MOE_LAUNCH("balance_gradient", s, balance_gradient<P>, dim3(g < most ? g : most), dim3(64 * kWaves), 0, s, a);
}

#define BALANCE_BY_E(E, CALL)            \
  do {                                   \
    const int per_ = ((E) + 63) / 64;    \
    if (per_ <= 1) CALL(1);              \
    else if (per_ <= 2) CALL(2);         \
    else if (per_ <= 4) CALL(4);         \
    else if (per_ <= 8) CALL(8);         \
    else if (per_ <= 16) CALL(16);       \
    else CALL(32);                       \
  } while (0)

}  // namespace

// Workspace: the row workgroups' sums, the finished counter, the counts.
size_t balance_workspace_bytes(int T, int k, int E) {
  return sizeof(float) * 2 * kRowGroups + 256 + sizeof(int32_t) * (size_t)count_groups(T, k) * (E + 1);
}

hipError_t launch_balance(const void* logits, int dtype, long long ld, int T, int E, int k, const int32_t* idx,
                          const uint8_t* keep, float* losses, int32_t* counts, int32_t* kept, void* ws,
                          hipStream_t s) {
  BalanceArgs a{};
  a.logits = logits;
  a.bf16 = dtype == 1;
  a.ld = ld;
  a.T = T;
  a.E = E;
  a.k = k;
  a.idx = idx;
  a.keep = keep;
  a.losses = losses;
  a.counts = counts;
  a.kept = kept;
  char* p = static_cast<char*>(ws);
  a.wsums = reinterpret_cast<float*>(p);
  a.done = reinterpret_cast<uint32_t*>(p + sizeof(float) * 2 * kRowGroups);
  a.wcounts = reinterpret_cast<int32_t*>(p + sizeof(float) * 2 * kRowGroups + 256);
  MOE_LAUNCH("balance_count", s, balance_count, dim3(count_groups(T, k)), dim3(256), 0, s, a);
#define ROWS(P) launch_rows<P>(a, s)
  BALANCE_BY_E(E, ROWS);
#undef ROWS
  return hipGetLastError();
}

hipError_t launch_balance_gradient(const void* logits, int dtype, long long ld, int T, int E, int k,
                                   const uint8_t* keep, const int32_t* counts, const int32_t* kept, const float* d,
                                   void* dx, hipStream_t s) {
  BalanceArgs a{};
  a.logits = logits;
  a.bf16 = dtype == 1;
  a.ld = ld;
  a.T = T;
  a.E = E;
  a.k = k;
  a.keep = keep;
  a.counts = const_cast<int32_t*>(counts);
  a.kept = const_cast<int32_t*>(kept);
  a.d = d;
  a.dx = dx;
#define GRAD(P) launch_grad<P>(a, s)
  BALANCE_BY_E(E, GRAD);
#undef GRAD
  return hipGetLastError();
}

}  // namespace moe
