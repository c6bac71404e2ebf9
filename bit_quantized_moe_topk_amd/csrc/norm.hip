// RMS norm with the residual's addition in front, its rows in float and in
// 8-bit blocks, and its gradients.
//
//   r = x + residual,  v = w r q,  q = 1 / sqrt(mean r^2 + eps)
//   dh = d_total + q (w dy - h q^2 mean(w dy h)),  dw = sum_t dy h q
//
// One pass: a row stays in registers between its sum and its results, eight
// neighbouring values a lane, so that 16 lanes hold an 8-bit block. The
// gradient needs two sums of a row, which are taken together; the weight's
// gradient stays in registers over the rows that a workgroup takes, and a second
// launch adds up the workgroups' parts in order. Bound by memory.
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
  bool vin, vout, vw;  // 16 bytes at a time: rows that come in, rows that go out, the weight
};

// Sums of N values over the W waves of a row, the same in each.
template <int W, int N>
__device__ inline void row_sums(float (&v)[N], float (*mem)[N], int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (W > 1) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, first = wave / W * W;
    constexpr int kWaves = W < 4 ? 4 : W;
    float(*m)[N] = mem + (turn & 1) * kWaves;
    turn ^= 1;  // (the next row's sums go elsewhere: one barrier a row)
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) m[wave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = m[first][i];
#pragma unroll
      for (int w = 1; w < W; ++w) s += m[first + w][i];
      v[i] = s;
    }
  }
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

template <int C, int W>
__device__ inline void load_weight(const NormArgs& a, float (&w)[C][8]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = Place<C, W>::col(c);
    if (a.wbf) load8<true>(a.weight, col, a.H, a.vw, w[c]);
    else load8<false>(a.weight, col, a.H, a.vw, w[c]);
  }
}

template <bool BF, int C, int W>
__global__ __launch_bounds__(threads_of(W)) void norm_forward(NormArgs a) {
  typedef Place<C, W> P;
  __shared__ float mem[2 * (W < 4 ? 4 : W)][1];
  constexpr int kSize = BF ? 2 : 4;
  const int nb = f8_blocks(a.H);
  float w[C][8];
  load_weight<C, W>(a, w);
  int turn = 0;
  for (int t0 = blockIdx.x * P::kRowsAtOnce; t0 < a.T; t0 += gridDim.x * P::kRowsAtOnce) {
    const int t = t0 + P::row();
    const bool there = t < a.T;
    float f[C][8], sum[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[c][i] = 0.f;
      const int col = P::col(c);
      if (there && col < a.H) {
        load8<BF>(static_cast<const char*>(a.x) + t * a.ldx * kSize, col, a.H, a.vin, f[c]);
        if (a.residual) {
          float g[8];
          load8<BF>(static_cast<const char*>(a.residual) + t * a.ldr * kSize, col, a.H, a.vin, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[c][i] += g[i];
        }
        if (a.total) store8<BF>(static_cast<char*>(a.total) + (size_t)t * a.H * kSize, col, a.H, a.vout, f[c]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] = fmaf(f[c][i], f[c][i], sum[0]);
    }
    row_sums<W, 1>(sum, mem, turn);
    const float q = 1.f / sqrtf(sum[0] / (float)a.H + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = P::col(c);
      if (!there || col >= nb * kF8Block) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = f[c][i] * q * w[c][i];
      if (a.y) store8<BF>(static_cast<char*>(a.y) + (size_t)t * a.H * kSize, col, a.H, a.vout, v);
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
  __shared__ float mem[2 * (W < 4 ? 4 : W)][2];
  constexpr int kSize = BF ? 2 : 4;
  float w[C][8], dw[C][8] = {};
  load_weight<C, W>(a, w);
  int turn = 0;
  for (int t0 = blockIdx.x * P::kRowsAtOnce; t0 < a.T; t0 += gridDim.x * P::kRowsAtOnce) {
    const int t = t0 + P::row();
    const bool there = t < a.T;
    float h[C][8], d[C][8], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = d[c][i] = 0.f;
      const int col = P::col(c);
      if (there && col < a.H) {
        load8<BF>(static_cast<const char*>(a.x) + t * a.ldx * kSize, col, a.H, a.vin, h[c]);
        load8<BF>(static_cast<const char*>(a.dy) + t * a.ldd * kSize, col, a.H, a.vin, d[c]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] = fmaf(h[c][i], h[c][i], sum[0]);
        sum[1] = fmaf(w[c][i] * d[c][i], h[c][i], sum[1]);
      }
    }
    row_sums<W, 2>(sum, mem, turn);
    const float q = 1.f / sqrtf(sum[0] / (float)a.H + a.eps);
    const float m = sum[1] / (float)a.H * q * q;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = P::col(c);
      if (!there || col >= a.H) continue;
      float g[8], v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 0.f;
      if (a.d_total) load8<BF>(static_cast<const char*>(a.d_total) + t * a.ldt * kSize, col, a.H, a.vin, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = fmaf(q, w[c][i] * d[c][i] - h[c][i] * m, g[i]);
        dw[c][i] = fmaf(d[c][i], h[c][i] * q, dw[c][i]);
      }
      store8<BF>(static_cast<char*>(a.dh) + (size_t)t * a.H * kSize, col, a.H, a.vout, v);
    }
  }
  if (!a.part) return;
  float* part = a.part + (size_t)(blockIdx.x * P::kRowsAtOnce + P::row()) * a.H;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = P::col(c);
    if (col < a.H) store8<false>(part, col, a.H, a.H % 4 == 0, dw[c]);
  }
}

// dweight[h] = the sum of n parts, 64 columns a workgroup, 16 runs of parts side by side.
__global__ __launch_bounds__(1024) void norm_parts(const float* __restrict__ part, int n, int H, float* __restrict__ dw) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
  float s = 0.f;
  const int per = (n + 15) / 16;
  if (col < H)
    for (int i = run * per; i < min(n, (run + 1) * per); ++i) s += part[(size_t)i * H + col];
  sums[run][lane] = s;
  __syncthreads();
  if (run || col >= H) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += sums[i][lane];
  dw[col] = s;
}

struct Shape {
  int C, W;
};
// Chunks of eight values a lane and waves a row.
Shape shape_of(int T, int H) {
  Shape s{1, 1};
  while (512 * s.C * s.W < H) {
    if (s.W < 4) s.W *= 2;
    else if (s.C < 4) s.C *= 2;
    else s.W *= 2;
  }
  return s;
}

constexpr int kParts = 1024;
int rows_at_once(const Shape& s) { return s.W < 4 ? 4 / s.W : 1; }
int grid_of(int T, const Shape& s, int most) {
  const int n = (T + rows_at_once(s) - 1) / rows_at_once(s);
  return n < most ? n : most;
}

bool all_vec(const void* p, long long ld, int size) { return !p || rows_vec(p, ld, size); }

#define NORM_FORMS(M, BF) \
  M(BF, 1, 1) M(BF, 1, 2) M(BF, 1, 4) M(BF, 2, 4) M(BF, 4, 4) M(BF, 4, 8) M(BF, 4, 16)

}  // namespace

size_t norm_workspace_bytes(int T, int H) {
  const Shape s = shape_of(T, H);
  return sizeof(float) * (size_t)H * grid_of(T, s, kParts / rows_at_once(s)) * rows_at_once(s);
}

hipError_t launch_norm(const void* x, int dtype, long long ldx, const void* residual, long long ldr, const void* weight,
                       int wdtype, float eps, int T, int H, void* total, void* y, uint8_t* codes, float* scales,
                       hipStream_t s) {
  const int size = dtype == 1 ? 2 : 4;
  NormArgs a{};
  a.x = x; a.ldx = ldx; a.residual = residual; a.ldr = ldr; a.weight = weight; a.wbf = wdtype == 1;
  a.eps = eps; a.T = T; a.H = H; a.total = total; a.y = y; a.codes = codes; a.scales = scales;
  a.vin = all_vec(x, ldx, size) && all_vec(residual, ldr, size);
  a.vout = all_vec(total, H, size) && all_vec(y, H, size);
  a.vw = rows_vec(weight, 0, 2);
  const Shape f = shape_of(T, H);
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
  const int size = dtype == 1 ? 2 : 4;
  NormArgs a{};
  a.x = h; a.ldx = ldh; a.dy = dy; a.ldd = ldd; a.d_total = d_total; a.ldt = ldt; a.weight = weight; a.wbf = wdtype == 1;
  a.eps = eps; a.T = T; a.H = H; a.dh = dh; a.part = dweight ? static_cast<float*>(ws) : nullptr;
  a.vin = all_vec(h, ldh, size) && all_vec(dy, ldd, size) && all_vec(d_total, ldt, size);
  a.vout = all_vec(dh, H, size);
  a.vw = rows_vec(weight, 0, 2);
  const Shape f = shape_of(T, H);
  const dim3 g(grid_of(T, f, kParts / rows_at_once(f)));
  if (T > 0) {
#define BACKWARD(BF, CC, WW) \
  if ((dtype == 1) == BF && f.C == CC && f.W == WW) \
    MOE_LAUNCH("norm_backward", s, (norm_backward<BF, CC, WW>), g, dim3(threads_of(WW)), 0, s, a);
    NORM_FORMS(BACKWARD, true)
    NORM_FORMS(BACKWARD, false)
#undef BACKWARD
  }
  if (dweight)
    MOE_LAUNCH("norm_parts", s, norm_parts, dim3((H + 63) / 64), dim3(1024), 0, s, a.part,
               T > 0 ? (int)g.x * rows_at_once(f) : 0, H, dweight);
  return hipGetLastError();
}

}  // namespace moe
