// Products of few 8-bit rows with an 8-bit matrix, and the products with the
// matrix turned (the gradient for the rows).
//
// Up to 16 rows of one group and 16 results a row per workgroup, on 16x16
// matrix-core tiles; four waves share the blocks of the contraction. Weights go
// from memory to registers. Bound by the matrix's bytes: each is read once per
// 16 rows.
#include "f8.h"

namespace moe {
namespace {

constexpr int kRows = 16;  // rows of a group per workgroup

// The group and rows of this workgroup: block x takes rows 16 x .. of the one
// matrix; with groups, block x works if row x is the first of a 16 of its group.
struct Unit {
  int e, s0, M;
};
__device__ inline Unit unit_of(const Mx4Args& a) {
  Unit u;
  if (!a.offsets) {
    u.e = 0;
    u.s0 = blockIdx.x * kRows;
    u.M = min(kRows, a.A - u.s0);
    return u;
  }
  u.s0 = blockIdx.x;
  u.e = mx4_group_of(a.offsets, a.E_tot, u.s0);
  u.M = 0;
  if (u.e < a.E_tot) {
    const int first = first_row(a, u.e);
    if (u.s0 >= first && (u.s0 - first) % kRows == 0) u.M = min(kRows, first_row(a, u.e + 1) - u.s0);
  }
  return u;
}

template <bool BACK, bool EXACT>
__global__ __launch_bounds__(256) void rows_product(F8Args a) {
  __shared__ floatx4_t part[4][64];
  const Unit u = unit_of(a);
  if (u.M <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.y * 16;
  const int row = max(mx4_row(a, u.s0 + min(r, u.M - 1)), 0);
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + (size_t)row * a.xb * kF8Block + 32 * g;
  const float* xs = a.xf + (size_t)row * a.xb;
  const int stored = BACK ? a.K : a.N;  // rows of the stored matrix
  const uint8_t* w = a.wc + (size_t)u.e * stored * a.wb * kF8Block;
  const float* ws = a.wf + (size_t)u.e * f8_blocks(stored) * a.wb;
  floatx4_t acc = {};
  for (int p = wave; p < a.xb; p += 4) {
    const uint4* xp = reinterpret_cast<const uint4*>(x + (size_t)p * kF8Block);
    int8v_t m;
    if constexpr (BACK) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = 0;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int c = min(p * kF8Block + 32 * g + 4 * i + z, a.K - 1);
          v[i] |= (uint32_t)w[(size_t)c * a.wb * kF8Block + n0 + r] << (8 * z);
        }
        m[i] = (int)v[i];
      }
    } else {
      const uint4* wp = reinterpret_cast<const uint4*>(w + ((size_t)min(n0 + r, a.N - 1) * a.wb + p) * kF8Block + 32 * g);
      m = f8_pair(wp[0], wp[1]);
    }
    const float s = xs[p] * ws[BACK ? (size_t)p * a.wb + n0 / kF8Block : (size_t)(n0 / kF8Block) * a.wb + p];
    const floatx4_t c = f8_products<EXACT>(m, f8_pair(xp[0], xp[1]));
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(c[i], s, acc[i]);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave || r >= u.M) return;
#pragma unroll
  for (int z = 1; z < 4; ++z) acc += part[z][lane];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 4 * g + i;
    if (n >= a.N) continue;
    const size_t at = (size_t)(u.s0 + r) * a.N + n;
    if (a.ydtype == 1) static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_bf16_bits(acc[i]);
    else static_cast<float*>(a.y)[at] = acc[i];
  }
}

}  // namespace

hipError_t launch_f8_product(const F8Args& a, hipStream_t s) {
  if (a.A >= (a.offsets ? 64 : 32) && f8_tiles_can(a)) return launch_f8_tiles(a, s);
  const dim3 g(a.offsets ? a.A : (a.A + kRows - 1) / kRows, (a.N + 15) / 16);
  if (a.back && a.exact) MOE_LAUNCH("f8_rows_back", s, (rows_product<true, true>), g, dim3(256), 0, s, a);
  else if (a.back) MOE_LAUNCH("f8_rows_back", s, (rows_product<true, false>), g, dim3(256), 0, s, a);
  else if (a.exact) MOE_LAUNCH("f8_rows", s, (rows_product<false, true>), g, dim3(256), 0, s, a);
  else MOE_LAUNCH("f8_rows", s, (rows_product<false, false>), g, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
