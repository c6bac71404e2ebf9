// RMS norm with the residual's addition in front, its rows in float and in
// 8-bit blocks, and its gradients.
//
//   r = x + residual,  v = w r q,  q = 1 / sqrt(mean r^2 + eps)
//   dh = d_total + q (w dy - h q^2 mean(w dy h)),  dw = sum_t dy h q
//
// One pass: a row stays in registers between its sum and its results, eight
// neighbouring values a lane, so that 16 lanes hold an 8-bit block. The
// gradient needs two sums of a row, which are taken together; the weight's
// gradient stays in registers, past 16,384 values in LDS, over the rows that a workgroup takes, and a second
// launch adds up the workgroups' parts in order: no atomics, so it repeats. Bound by memory:
// 8,192 rows of 2,048 bf16 values with a residual to total, rows, 8-bit rows and scales, 25.6 to 28.4 us
// (5.5 TB/s with part of the rows from cache; a copy reaches 5.1); the gradient at float32 with a d_total, 8,192 rows of
// 4,096, 95 us (5.7 TB/s) and 4 for the parts. A few rows take 4 to 5 us a launch.
#include "f8.h"
#include "norm.h"

namespace moe {
namespace {

struct NormArgs {
  const void *x, *residual, *weight, *dy, *d_total;
  long long ldx, ldr, ldd, ldt;
  int T, H, wbf;
  float eps;
  void *total, *y, *dh;
  uint8_t* codes;
  float* scales;
  float* part;
};

__device__ inline double wave_sum(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sums of N values over the W waves of a row, the same in each.
template <int W, int N, typename F>
__device__ inline void row_sums(F (&v)[N], F (*mem)[N], int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (W > 1) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, first = wave / W * W;
    constexpr int kWaves = W < 4 ? 4 : W;
    F(*m)[N] = mem + (turn & 1) * kWaves;
    turn ^= 1;  // (the next row's sums go elsewhere: one barrier a row)
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) m[wave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      F s = m[first][i];
#pragma unroll
      for (int w = 1; w < W; ++w) s += m[first + w][i];
      v[i] = s;
    }
  }
}

// 1 / sqrt(m) in 64 bits: one step from the 32-bit instruction's, where that holds.
__device__ inline double inverse_root(double m) {
  if (!(m > 0x1p-100 && m < 0x1p100)) return 1.0 / sqrt(m);
  const double y = __builtin_amdgcn_rsqf((float)m);
  return y * (1.5 - 0.5 * m * y * y);
}

constexpr int threads_of(int W) { return W < 4 ? 256 : 64 * W; }

template <int C, int W>
struct Place {
  static constexpr int kThreads = threads_of(W);
  static constexpr int kRowsAtOnce = kThreads / (64 * W);  // rows in flight per workgroup
  __device__ static int lane() { return threadIdx.x % (64 * W); }
  __device__ static int col(int c) { return 8 * (c * 64 * W + lane()); }
  __device__ static int row() { return threadIdx.x / (64 * W); }
};

__device__ inline void weight_at(const NormArgs& a, int col, float (&w)[8]) {
  if (a.wbf) load8<true>(a.weight, col, a.H, w);
  else load8<false>(a.weight, col, a.H, w);
}

// (Spelled out: as calls of weight_at the compiler leaves these loads within the loop over rows, 33.4 us for 27.8.)
template <int C, int W>
__device__ inline void load_weight(const NormArgs& a, float (&w)[C][8]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = Place<C, W>::col(c);
    if (a.wbf) load8<true>(a.weight, col, a.H, w[c]);
    else load8<false>(a.weight, col, a.H, w[c]);
  }
}

template <bool BF, int C, int W>
__global__ __launch_bounds__(threads_of(W)) void norm_forward(NormArgs a) {
  typedef Place<C, W> P;
  __shared__ double mem[2 * (W < 4 ? 4 : W)][1];
  constexpr int kSize = BF ? 2 : 4;
  const int nb = f8_blocks(a.H);
  float w[C][8];
  load_weight<C, W>(a, w);
  int turn = 0;
  for (int t0 = blockIdx.x * P::kRowsAtOnce; t0 < a.T; t0 += gridDim.x * P::kRowsAtOnce) {
    const int t = t0 + P::row();
    const bool there = t < a.T;
    float f[C][8], part = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[c][i] = 0.f;
      const int col = P::col(c);
      if (there && col < a.H) {
        load8<BF>(static_cast<const char*>(a.x) + t * a.ldx * kSize, col, a.H, f[c]);
        if (a.residual) {
          float g[8];
          load8<BF>(static_cast<const char*>(a.residual) + t * a.ldr * kSize, col, a.H, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[c][i] += g[i];
        }
        if (a.total) store8<BF>(static_cast<char*>(a.total) + (size_t)t * a.H * kSize, col, a.H, f[c]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) part = fmaf(f[c][i], f[c][i], part);
    }
    // From a lane's sum on in 64 bits, and the factor as two 32-bit parts: a value is off by its last rounding, and a
    // block's scale hardly ever, which leaves a few codes in a million on the other side of a border.
    double sum[1] = {part};
    row_sums<W, 1>(sum, mem, turn);
    const double root = inverse_root(sum[0] / a.H + (double)a.eps);
    const float q = (float)root, ql = fabsf(q) < INFINITY ? (float)(root - (double)q) : 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = P::col(c);
      if (!there || col >= nb * kF8Block) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = f[c][i] * q;
        v[i] = fmaf(u, w[c][i], fmaf(f[c][i], ql, fmaf(f[c][i], q, -u)) * w[c][i]);
        v[i] = v[i] != v[i] ? u * w[c][i] : v[i];  // (an infinite weight is the first part's alone: the second may be 0)
      }
      if (a.y) store8<BF>(static_cast<char*>(a.y) + (size_t)t * a.H * kSize, col, a.H, v);
      if (a.codes) {
        // past the row's end there is nothing, whatever q is
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = col + i < a.H ? v[i] : 0.f;
        float sc;
        const uint2 u = f8_codes(v, f8_top16(v), &sc);
        *reinterpret_cast<uint2*>(a.codes + (size_t)t * nb * kF8Block + col) = u;
        if ((threadIdx.x & 15) == 0) a.scales[(size_t)t * nb + col / kF8Block] = sc;
      }
    }
  }
}

template <bool BF, int C, int W>
__global__ __launch_bounds__(threads_of(W)) void norm_backward(NormArgs a) {
  typedef Place<C, W> P;
  __shared__ double mem[2 * (W < 4 ? 4 : W)][2];
  constexpr int kSize = BF ? 2 : 4;
  // A lane's part of the weight, h, dy and the weight's gradient stay in registers, but where a workgroup has 1,024 threads, and so 128
  // registers each: there the gradient is in LDS, and the rest is read again for the results (1,024 bf16 rows of 20,000 46 us, of
  // 32,768 87; held, with 75 registers of a lane spilled, 103 and 142).
  constexpr bool kHold = W < 16;
  constexpr int kKept = kHold ? C : 1;
  __shared__ __attribute__((aligned(16))) float far[kHold ? 1 : P::kThreads * C * 8];
  float held[kKept][8], dw[kKept][8] = {};
  auto place = [&](int c) { return far + 8 * (c * P::kThreads + threadIdx.x); };
  // f(chunk), chunks unrolled only where they are held
  auto chunks = [&](auto f) __attribute__((always_inline)) {
    if constexpr (kHold) {
#pragma unroll
      for (int c = 0; c < C; ++c) f(c);
    } else {
#pragma unroll 1
      for (int c = 0; c < C; ++c) f(c);
    }
  };
  if constexpr (kHold) load_weight<C, W>(a, held);
  else chunks([&](int c) __attribute__((always_inline)) { store8<false>(place(c), 0, 8, dw[0]); });
  auto weight = [&](int c, float (&w)[8]) __attribute__((always_inline)) {
    if constexpr (!kHold) return weight_at(a, P::col(c), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = held[kHold ? c : 0][i];
  };
  int turn = 0;
  for (int t0 = blockIdx.x * P::kRowsAtOnce; t0 < a.T; t0 += gridDim.x * P::kRowsAtOnce) {
    const int t = t0 + P::row();
    const bool there = t < a.T;
    float h[kKept][8], d[kKept][8], sum[2] = {0.f, 0.f};
    auto load_row = [&](int c) __attribute__((always_inline)) {
      const int at = kHold ? c : 0, col = P::col(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[at][i] = d[at][i] = 0.f;
      if (there && col < a.H) {
        load8<BF>(static_cast<const char*>(a.x) + t * a.ldx * kSize, col, a.H, h[at]);
        load8<BF>(static_cast<const char*>(a.dy) + t * a.ldd * kSize, col, a.H, d[at]);
      }
    };
    chunks([&](int c) __attribute__((always_inline)) {
      const int at = kHold ? c : 0;
      load_row(c);
      float w[8];
      weight(c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] = fmaf(h[at][i], h[at][i], sum[0]);
        sum[1] = fmaf(w[i] * d[at][i], h[at][i], sum[1]);
      }
    });
    // From a lane's sums on in 64 bits, as in the forward call, which norms rows whose sum of squares passes 2^128; rounded once, as an error
    // of q is one of the whole row.
    double all[2] = {sum[0], sum[1]};
    row_sums<W, 2>(all, mem, turn);
    const double root = inverse_root(all[0] / a.H + (double)a.eps);
    const float q = (float)root, m = (float)(all[1] / a.H * root * root);
    chunks([&](int c) __attribute__((always_inline)) {
      const int col = P::col(c), at = kHold ? c : 0;
      if (!there || col >= a.H) return;
      if constexpr (!kHold) {
        load_row(c);
        load8<false>(place(c), 0, 8, dw[0]);
      }
      float g[8], v[8], w[8];
      weight(c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 0.f;
      if (a.d_total) load8<BF>(static_cast<const char*>(a.d_total) + t * a.ldt * kSize, col, a.H, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = fmaf(q, w[i] * d[at][i] - h[at][i] * m, g[i]);
        dw[at][i] = fmaf(d[at][i], h[at][i] * q, dw[at][i]);
      }
      store8<BF>(static_cast<char*>(a.dh) + (size_t)t * a.H * kSize, col, a.H, v);
      if constexpr (!kHold) store8<false>(place(c), 0, 8, dw[0]);
    });
  }
  if (!a.part) return;
  // the workgroup's rows in flight, then its part
  if constexpr (P::kRowsAtOnce > 1) {
    __shared__ __attribute__((aligned(16))) float rows[P::kRowsAtOnce - 1][8 * 64 * W * C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (P::row() > 0) store8<false>(rows[P::row() - 1], P::col(c), 1 << 30, dw[c]);
    __syncthreads();
    if (P::row() > 0) return;
#pragma unroll
    for (int z = 0; z + 1 < P::kRowsAtOnce; ++z)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] += rows[z][P::col(c) + i];
  }
  float* part = a.part + (size_t)blockIdx.x * a.H;
  chunks([&](int c) __attribute__((always_inline)) {
    const int col = P::col(c);
    if (col >= a.H) return;
    if constexpr (!kHold) load8<false>(place(c), 0, 8, dw[0]);
    store8<false>(part, col, a.H, dw[kHold ? c : 0]);
  });
}

// dweight[h] = the sum of n parts, 32 columns a workgroup, 32 runs of parts side by side, eight loads at once.
__global__ __launch_bounds__(1024) void norm_parts(const float* __restrict__ part, int n, int H, float* __restrict__ dw) {
  __shared__ float sums[32][33];
  const int c = threadIdx.x & 31, run = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  const int per = (n + 31) / 32, end = min(n, (run + 1) * per);
  float s = 0.f;
  for (int i = run * per; i < end && col < H; i += 8) {
    float v[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) v[z] = part[(size_t)min(i + z, end - 1) * H + col];
#pragma unroll
    for (int z = 0; z < 8; ++z) s += i + z < end ? v[z] : 0.f;
  }
  sums[run][c] = s;
  __syncthreads();
  if (run || col >= H) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) s += sums[i][c];
  dw[col] = s;
}

struct Shape {
  int C, W;
};
// Chunks of eight values a lane and waves a row: up to four waves before a second chunk, which keeps a row's loads short of one
// another's way. Measured, waves first against chunks first: 8,192 rows of 2,048 in bf16 25.5 us against 29.6, of 4,096 61 against
// 79, 64 rows of 2,048 4.7 against 7.7. (More waves at once would leave fewer rows a workgroup for the weight's gradient.)
Shape shape_of(int H) {
  Shape s{1, 1};
  while (512 * s.C * s.W < H) {
    if (s.W < 4) s.W *= 2;
    else if (s.C < 4) s.C *= 2;
    else s.W *= 2;
  }
  return s;
}

// Most workgroups of the gradient, each of which leaves a row of parts. Gradient and parts, float32: 8,192 rows of 2,048 with 128
// 86 us, 256 49, 512 35, 1,024 37, 2,048 40; of 4,096 165, 97, 83, 84, 90.
constexpr int kParts = 512;
int rows_at_once(const Shape& s) { return s.W < 4 ? 4 / s.W : 1; }
int grid_of(int T, const Shape& s, int most) {
  const int n = (T + rows_at_once(s) - 1) / rows_at_once(s);
  return n < most ? n : most;
}

#define NORM_FORMS(M, BF) \
  M(BF, 1, 1) M(BF, 1, 2) M(BF, 1, 4) M(BF, 2, 4) M(BF, 4, 4) M(BF, 4, 8) M(BF, 4, 16)

}  // namespace

size_t norm_workspace_bytes(int T, int H) {
  const Shape s = shape_of(H);
  return sizeof(float) * (size_t)H * grid_of(T, s, kParts);
}

hipError_t launch_norm(const void* x, int dtype, long long ldx, const void* residual, long long ldr, const void* weight,
                       int wdtype, float eps, int T, int H, void* total, void* y, uint8_t* codes, float* scales,
                       hipStream_t s) {
  NormArgs a{};
  a.x = x; a.ldx = ldx; a.residual = residual; a.ldr = ldr; a.weight = weight; a.wbf = wdtype == 1;
  a.eps = eps; a.T = T; a.H = H; a.total = total; a.y = y; a.codes = codes; a.scales = scales;
  const Shape f = shape_of(H);
  const dim3 g(grid_of(T, f, 8 * device_cus()));
#define FORWARD(BF, CC, WW) \
  if ((dtype == 1) == BF && f.C == CC && f.W == WW) \
    MOE_LAUNCH("norm", s, (norm_forward<BF, CC, WW>), g, dim3(threads_of(WW)), 0, s, a);
  NORM_FORMS(FORWARD, true)
  NORM_FORMS(FORWARD, false)
#undef FORWARD
  return hipGetLastError();
}

hipError_t launch_norm_backward(const void* dy, long long ldd, const void* h, long long ldh, int dtype, const void* weight,
                                int wdtype, const void* d_total, long long ldt, float eps, int T, int H, void* dh,
                                float* dweight, void* ws, hipStream_t s) {
  NormArgs a{};
  a.x = h; a.ldx = ldh; a.dy = dy; a.ldd = ldd; a.d_total = d_total; a.ldt = ldt; a.weight = weight; a.wbf = wdtype == 1;
  a.eps = eps; a.T = T; a.H = H; a.dh = dh; a.part = dweight ? static_cast<float*>(ws) : nullptr;
  const Shape f = shape_of(H);
  const dim3 g(grid_of(T, f, kParts));
  if (T > 0) {
#define BACKWARD(BF, CC, WW) \
  if ((dtype == 1) == BF && f.C == CC && f.W == WW) \
    MOE_LAUNCH("norm_backward", s, (norm_backward<BF, CC, WW>), g, dim3(threads_of(WW)), 0, s, a);
    NORM_FORMS(BACKWARD, true)
    NORM_FORMS(BACKWARD, false)
#undef BACKWARD
  }
  if (dweight)
    MOE_LAUNCH("norm_parts", s, norm_parts, dim3((H + 31) / 32), dim3(1024), 0, s, a.part, T > 0 ? (int)g.x : 0, H, dweight);
  return hipGetLastError();
}

}  // namespace moe
