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
// many values. Bound by those bytes; small batches, which one workgroup counts
// and sums in one launch, by its latency.
//
// Sums are float32 in a fixed order (per wave over its tokens, then over the
// waves in order), counts are integers: results do not vary from run to run.
#include "balance.h"
#include "gemv.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int kWaves = 4;         // tokens in flight per workgroup
constexpr int kSmallWaves = 16;   // the same of the one-launch form
// The one-launch form's most tokens, ids and logits: all pass through one CU, which soon takes longer than two launches
// on the GPU (k = 10; one launch against two: 16 x 512 5.6 us against 8.8, 64 x 512 10.7 against 9.1, 128 x 512 17.7
// against 9.1, 128 x 2,048 45 against 15; 64 x 512 with k = 128 11.1 against 10.3), but a launch less is 3 us of the
// host's time, which bounds a small call.
constexpr int kSmallT = 128, kSmallIds = 4096, kSmallLogits = 1 << 15;
// Ids per counting workgroup: every workgroup of the pass adds up all their counts, so few of them (forward, 8,192
// tokens x 10: 18.6 us, with 512 ids 20.5, with 8,192 18.2), and not too few (1,000 x 8: 9.3 us, with 1,024 ids 8.5,
// with 8,192 10.2).
constexpr int kCountIds = 4096;
constexpr int kCountGroups = 64;  // most counting workgroups
// Most workgroups of the pass over the logits (65,536 x 512: 53 us, with 512 63, with 256 91; 8,192 x 512: 18.8, 18.3 and
// 20.5).
constexpr int kRowGroups = 1024;
constexpr int kLines = 16;        // counters of finished workgroups, a line each, before the last one

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
  uint32_t* done;       // [kLines + 1], 32 words apart
};

// Columns of a lane: P of them, one at a time (lane + 64 i in slot i), or with
// VEC in fours (4 (lane + 64 (i / 4)) + i % 4).
template <bool VEC>
__device__ inline int column(int i) {
  const int lane = threadIdx.x & 63;
  return VEC ? 4 * (lane + 64 * (i >> 2)) + (i & 3) : lane + 64 * i;
}

// A token's logits as they lie in memory: P dwords, or P / 2 for bf16 in fours.
template <int P, bool VEC>
struct RawRow {
  uint32_t v[P];
};
template <int P, bool VEC>
__device__ inline void load_raw(const BalanceArgs& a, int t, RawRow<P, VEC>& raw) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < P; i += 4) {
      const int c = column<VEC>(i);
      if (c >= a.E) continue;
      if (a.bf16) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + (size_t)t * a.ld + c);
        raw.v[i] = u.x << 16;
        raw.v[i + 1] = u.x & 0xFFFF0000u;
        raw.v[i + 2] = u.y << 16;
        raw.v[i + 3] = u.y & 0xFFFF0000u;
      } else {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const float*>(a.logits) + (size_t)t * a.ld + c);
        raw.v[i] = u.x;
        raw.v[i + 1] = u.y;
        raw.v[i + 2] = u.z;
        raw.v[i + 3] = u.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = column<VEC>(i);
      if (c >= a.E) continue;
      const size_t at = (size_t)t * a.ld + c;
      raw.v[i] = a.bf16 ? (uint32_t)static_cast<const uint16_t*>(a.logits)[at] << 16
                        : __float_as_uint(static_cast<const float*>(a.logits)[at]);
    }
  }
}

__device__ inline float wave_maxf(float v) {
  v = fmaxf(v, __uint_as_float(dpp(__float_as_uint(v), 0xB1)));
  v = fmaxf(v, __uint_as_float(dpp(__float_as_uint(v), 0x4E)));
  v = fmaxf(v, __uint_as_float(dpp(__float_as_uint(v), 0x141)));
  v = fmaxf(v, __uint_as_float(dpp(__float_as_uint(v), 0x140)));
  const float r0 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 0));
  const float r1 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 16));
  const float r2 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 32));
  const float r3 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 48));
  return fmaxf(fmaxf(r0, r1), fmaxf(r2, r3));
}

// exp(x - max) of a token's logits; *lse and 1 / sum. A token whose logits are
// all -inf has no distribution: p is 0 and lse 0.
template <int P, bool VEC>
__device__ inline void softmax_row(const BalanceArgs& a, const RawRow<P, VEC>& raw, float (&x)[P], float* lse,
                                   float* inv) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    x[i] = column<VEC>(i) < a.E ? __uint_as_float(raw.v[i]) : -INFINITY;
    top = fmaxf(top, x[i]);
  }
  top = wave_maxf(top);
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

// f of this lane's columns, from the finished counts.
template <int P, bool VEC>
__device__ inline void load_share(const int32_t* counts, int n, const BalanceArgs& a, float (&f)[P]) {
  const float total = (float)n * (float)a.k;
#pragma unroll
  for (int i = 0; i < P; ++i)
    f[i] = column<VEC>(i) < a.E && n > 0 ? (float)counts[column<VEC>(i)] / total : 0.f;
}

// Counts the ids of tokens [t0, t1) into the LDS histogram h[0 .. E], their
// kept tokens in h[E]; the workgroup's threads together, eight loads in flight each.
__device__ inline void count_ids(const BalanceArgs& a, int t0, int t1, int32_t* h) {
  const int tid = threadIdx.x, n = blockDim.x;
  for (int e = tid; e <= a.E; e += n) h[e] = 0;
  __syncthreads();
  const long long end = (long long)t1 * a.k;
  for (long long i = (long long)t0 * a.k + tid; i < end; i += 8 * n) {
    int e[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      const long long j = i + z * n;
      e[z] = j < end ? a.idx[j] : -1;
    }
#pragma unroll
    for (int z = 0; z < 8; ++z)
      if ((unsigned)e[z] < (unsigned)a.E && (!a.keep || a.keep[(int)((unsigned)(i + z * n) / (unsigned)a.k)]))
        atomicAdd(&h[e[z]], 1);
  }
  if (a.keep) {
    int kept = 0;
    for (int t = t0 + tid; t < t1; t += n) kept += a.keep[t] ? 1 : 0;
    if (kept) atomicAdd(&h[a.E], kept);
  } else if (tid == 0) {
    h[a.E] = t1 - t0;
  }
  __syncthreads();
}

// The sums of f . p_t and lse_t^2 over tokens t0, t0 + step, ..; the next
// token's logits are on their way while one is summed.
template <int P, bool VEC>
__device__ inline void sum_rows(const BalanceArgs& a, const float (&f)[P], int t0, int step, float* fp, float* zz) {
  *fp = 0.f;
  *zz = 0.f;
  RawRow<P, VEC> raw, next;
  int t = t0;
  if (t < a.T) load_raw(a, t, raw);
  while (t < a.T) {
    const int tn = t + step;
    if (tn < a.T) load_raw(a, tn, next);
    if (!a.keep || a.keep[t]) {
      float x[P], lse, inv, dot = 0.f;
      softmax_row<P, VEC>(a, raw, x, &lse, &inv);
#pragma unroll
      for (int i = 0; i < P; ++i) dot = fmaf(f[i], x[i], dot);
      *fp += wave_sum(dot) * inv;
      *zz += lse * lse;
    }
    raw = next;
    t = tn;
  }
}

__device__ inline void write_losses(const BalanceArgs& a, float fp, float zz, int n) {
  a.losses[0] = n ? fp * ((float)a.E / (float)n) : 0.f;
  a.losses[1] = n ? zz / (float)n : 0.f;
}

// A small batch in one workgroup: counts, then the pass.
template <int P, bool VEC>
__global__ __launch_bounds__(64 * kSmallWaves) void balance_small(BalanceArgs a) {
  __shared__ int32_t cnt[MOE_MAX_E_DEV + 1];
  __shared__ float ws[kSmallWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  count_ids(a, 0, a.T, cnt);
  for (int e = tid; e <= a.E; e += 64 * kSmallWaves) {
    if (e < a.E) a.counts[e] = cnt[e];
    else *a.kept = cnt[e];
  }
  const int n = cnt[a.E];
  float f[P], fp, zz;
  load_share<P, VEC>(cnt, n, a, f);
  sum_rows<P, VEC>(a, f, wave, kSmallWaves, &fp, &zz);
  if (lane == 0) {
    ws[wave][0] = fp;
    ws[wave][1] = zz;
  }
  __syncthreads();
  if (tid == 0) {
    fp = zz = 0.f;
    for (int w = 0; w < kSmallWaves; ++w) {
      fp += ws[w][0];
      zz += ws[w][1];
    }
    write_losses(a, fp, zz, n);
  }
}

// Counting workgroup b of G: the ids of tokens [b T / G, (b + 1) T / G).
__global__ __launch_bounds__(256) void balance_count(BalanceArgs a) {
  __shared__ int32_t h[MOE_MAX_E_DEV + 1];
  const int G = gridDim.x, b = blockIdx.x;
  count_ids(a, (int)((long long)b * a.T / G), (int)((long long)(b + 1) * a.T / G), h);
  for (int e = threadIdx.x; e <= a.E; e += 256) a.wcounts[(size_t)b * (a.E + 1) + e] = h[e];
  if (b == 0 && threadIdx.x <= kLines) a.done[32 * threadIdx.x] = 0u;
}

// Whether this is the last workgroup: each counts itself on one of kLines
// lines, the last of a line counts the line. (One counter for all of them took
// 20 us of the pass over 8,192 tokens: adds to one address queue up.) The
// workgroup's sums are stored past the caches, and have arrived, before.
__device__ inline bool last_workgroup(uint32_t* done) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  const int G = gridDim.x, line = blockIdx.x % kLines;
  const uint32_t of = (uint32_t)((G - line + kLines - 1) / kLines), lines = (uint32_t)min(G, kLines);
  if (__hip_atomic_fetch_add(done + 32 * line, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != of - 1) return false;
  return __hip_atomic_fetch_add(done + 32 * kLines, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == lines - 1;
}

// Pass over the logits. Every workgroup adds up the counting workgroups'
// counts (the first also writes them out); the last one to finish adds up the
// workgroups' sums in order.
template <int P, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void balance_rows(BalanceArgs a, int G) {
  __shared__ int32_t cnt[MOE_MAX_E_DEV + 1];
  __shared__ float ws[kWaves][2];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= a.E; e += 64 * kWaves) {
    int c = 0;
#pragma unroll 8
    for (int b = 0; b < G; ++b) c += a.wcounts[(size_t)b * (a.E + 1) + e];
    cnt[e] = c;
    if (blockIdx.x == 0) {
      if (e < a.E) a.counts[e] = c;
      else *a.kept = c;
    }
  }
  __syncthreads();
  const int n = cnt[a.E];
  float f[P], fp, zz;
  load_share<P, VEC>(cnt, n, a, f);
  sum_rows<P, VEC>(a, f, blockIdx.x * kWaves + wave, gridDim.x * kWaves, &fp, &zz);
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
    last = last_workgroup(a.done);
  }
  __syncthreads();
  if (!last || wave) return;
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
  for (int b = lane; b < (int)gridDim.x; b += 64) {
    s0 += __hip_atomic_load(&a.wsums[2 * b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s1 += __hip_atomic_load(&a.wsums[2 * b + 1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  s0 = wave_sum(s0);
  s1 = wave_sum(s1);
  if (lane == 0) write_losses(a, s0, s1, n);
}

template <int P, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void balance_gradient(BalanceArgs a) {
  const int wave = threadIdx.x >> 6, step = gridDim.x * kWaves;
  int t = blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  RawRow<P, VEC> raw, next;
  load_raw(a, t, raw);
  const int n = *a.kept;
  float f[P];
  load_share<P, VEC>(a.counts, n, a, f);
  const float cb = n ? a.d[0] * ((float)a.E / (float)n) : 0.f, cz = n ? a.d[1] * (2.f / (float)n) : 0.f;
  for (;;) {
    const int tn = t + step;
    if (tn < a.T) load_raw(a, tn, next);
    float x[P], lse = 0.f, inv = 0.f, dot = 0.f;
    const bool keep = !a.keep || a.keep[t];
    if (keep) {
      softmax_row<P, VEC>(a, raw, x, &lse, &inv);
#pragma unroll
      for (int i = 0; i < P; ++i) dot = fmaf(f[i], x[i], dot);
      dot = wave_sum(dot) * inv;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = keep ? x[i] * inv * fmaf(cb, f[i] - dot, cz * lse) : 0.f;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < P; i += 4) {
        const int c = column<VEC>(i);
        if (c >= a.E) continue;
        if (a.bf16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dx) + (size_t)t * a.E + c) =
              make_uint2(f32_to_bf16_bits(x[i]) | f32_to_bf16_bits(x[i + 1]) << 16,
                         f32_to_bf16_bits(x[i + 2]) | f32_to_bf16_bits(x[i + 3]) << 16);
        else
          *reinterpret_cast<float4*>(static_cast<float*>(a.dx) + (size_t)t * a.E + c) =
              make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = column<VEC>(i);
        if (c >= a.E) continue;
        if (a.bf16) static_cast<uint16_t*>(a.dx)[(size_t)t * a.E + c] = (uint16_t)f32_to_bf16_bits(x[i]);
        else static_cast<float*>(a.dx)[(size_t)t * a.E + c] = x[i];
      }
    }
    if (tn >= a.T) break;
    raw = next;
    t = tn;
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

template <int P, bool VEC>
void launch_rows(const BalanceArgs& a, hipStream_t s) {
  if (a.T <= kSmallT && (long long)a.T * a.k <= kSmallIds && (long long)a.T * a.E <= kSmallLogits) {
    MOE_LAUNCH("balance_small", s, (balance_small<P, VEC>), dim3(1), dim3(64 * kSmallWaves), 0, s, a);
    return;
  }
  const int G = count_groups(a.T, a.k);
  MOE_LAUNCH("balance_count", s, balance_count, dim3(G), dim3(256), 0, s, a);
  MOE_LAUNCH("balance_rows", s, (balance_rows<P, VEC>), dim3(row_groups(a.T)), dim3(64 * kWaves), 0, s, a, G);
}
template <int P, bool VEC>
void launch_grad(const BalanceArgs& a, hipStream_t s) {
  const int g = (a.T + kWaves - 1) / kWaves, most = 8 * device_cus();
  MOE_LAUNCH("balance_gradient", s, (balance_gradient<P, VEC>), dim3(g < most ? g : most), dim3(64 * kWaves), 0, s, a);
}

// Columns per lane for E, in fours where every row starts and ends on a group of four.
#define BALANCE_BY_E(E, VEC4, CALL)               \
  do {                                            \
    const int per_ = ((E) + 63) / 64;             \
    if (VEC4) {                                   \
      if (per_ <= 4) CALL(4, true);               \
      else if (per_ <= 8) CALL(8, true);          \
      else if (per_ <= 16) CALL(16, true);        \
      else CALL(32, true);                        \
    } else if (per_ <= 1) CALL(1, false);         \
    else if (per_ <= 2) CALL(2, false);           \
    else if (per_ <= 4) CALL(4, false);           \
    else if (per_ <= 8) CALL(8, false);           \
    else if (per_ <= 16) CALL(16, false);         \
    else CALL(32, false);                         \
  } while (0)

// E > 128: fewer experts fill the wave better one at a time (8,192 x 128 float32, fours against ones: 12.0 us against 11.1,
// the gradient 6.9 against 5.5; 8,192 x 512: 16.0 against 16.3, 14.2 against 13.2; 65,536 x 512: 53 against 55 and 53
// against 56, bf16 52 against 72 and 47 against 56; 8,192 x 2,048: 41 against 44, 46 against 71).
bool in_fours(const void* p, long long ld, const void* q, int E, int bf16) {
  const unsigned size = bf16 ? 8 : 16;
  return E > 128 && E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % size == 0 &&
         reinterpret_cast<uintptr_t>(q) % size == 0;
}

}  // namespace

// Workspace: the row workgroups' sums, the finished counter, the counts.
constexpr size_t kSumBytes = sizeof(float) * 2 * kRowGroups, kDoneBytes = 128 * (kLines + 1);
size_t balance_workspace_bytes(int T, int k, int E) {
  return kSumBytes + kDoneBytes + sizeof(int32_t) * (size_t)count_groups(T, k) * (E + 1);
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
  a.done = reinterpret_cast<uint32_t*>(p + kSumBytes);
  a.wcounts = reinterpret_cast<int32_t*>(p + kSumBytes + kDoneBytes);
#define ROWS(P, V) launch_rows<P, V>(a, s)
  BALANCE_BY_E(E, in_fours(logits, ld, nullptr, E, a.bf16), ROWS);
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
#define GRAD(P, V) launch_grad<P, V>(a, s)
  BALANCE_BY_E(E, in_fours(logits, ld, dx, E, a.bf16), GRAD);
#undef GRAD
  return hipGetLastError();
}

}  // namespace moe
