// Products of few 8-bit rows with an 8-bit matrix, and the products with the
// matrix turned (the gradient for the rows).
//
// Up to 16 rows of one group and 16 or 32 results a row per workgroup, on 16x16
// matrix-core tiles; four waves share the blocks of the contraction. Weights go
// from memory to registers, no LDS before the waves' sums. Bound by one chain of loads, products and sums while there is a
// workgroup a CU (one row, [1024, 2048], 3.9 us, of which a launch is about 3), then by the matrix's bytes, which are read once per
// 16 rows: 16 rows of [8192, 8192] 22 us, 3.1 TB/s.
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

// Lane (r, g) holds chunks 2 g and 2 g + 1 of a block of matrix row n0 + 16 j + r and of x's row r. A wave asks for its next
// kAhead blocks at once: with a few rows the time is the chain from the group's offsets over its loads to the sums.
template <bool EXACT, int NT>
__global__ __launch_bounds__(256) void rows_product(F8Args a) {
  constexpr int kAhead = 4;
  __shared__ floatx4_t part[4][NT][64];
  const Unit u = unit_of(a);
  if (u.M <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.y * 16 * NT;
  const int row = max(mx4_row(a, u.s0 + min(r, u.M - 1)), 0);
  const uint4* xp = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.x) + (size_t)row * a.xb * kF8Block + 32 * g);
  const float* xs = a.xf + (size_t)row * a.xb;
  const uint4* wp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    wp[j] = reinterpret_cast<const uint4*>(a.wc + ((size_t)u.e * a.N + min(n0 + 16 * j + r, a.N - 1)) * a.wb * kF8Block + 32 * g);
  const float* ws = a.wf + ((size_t)u.e * f8_blocks(a.N) + n0 / kF8Block) * a.wb;  // (16 NT rows are of one block of rows)
  floatx4_t acc[NT] = {};
  for (int p0 = wave; p0 < a.xb; p0 += 4 * kAhead) {
    uint4 w[kAhead][NT][2], x[kAhead][2];
    float s[kAhead];
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      const int p = min(p0 + 4 * z, a.xb - 1);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) w[z][j][i] = wp[j][8 * (size_t)p + i];
    }
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      const int p = min(p0 + 4 * z, a.xb - 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) x[z][i] = xp[8 * (size_t)p + i];
      s[z] = xs[p] * ws[p];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      if (p0 + 4 * z >= a.xb) break;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const floatx4_t c = f8_products<EXACT>(f8_pair(w[z][j][0], w[z][j][1]), f8_pair(x[z][0], x[z][1]));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(c[i], s[z], acc[j][i]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  // wave j brings results 16 j on
  if (wave >= NT || r >= u.M) return;
  floatx4_t y = part[0][wave][lane];
#pragma unroll
  for (int z = 1; z < 4; ++z) y += part[z][wave][lane];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 16 * wave + 4 * g + i;
    if (n >= a.N) continue;
    const size_t at = (size_t)(u.s0 + r) * a.N + n;
    if (a.ydtype == 1) static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_bf16_bits(y[i]);
    else static_cast<float*>(a.y)[at] = y[i];
  }
}

// The same with the matrix turned, for what the tiles cannot address (past 4 GiB of rows, or of one matrix): a lane
// gathers its codes a byte at a time.
template <bool EXACT>
__global__ __launch_bounds__(256) void rows_back(F8Args a) {
  __shared__ floatx4_t part[4][64];
  const Unit u = unit_of(a);
  if (u.M <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4, n0 = blockIdx.y * 16;
  const int row = max(mx4_row(a, u.s0 + min(r, u.M - 1)), 0);
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + (size_t)row * a.xb * kF8Block + 32 * g;
  const uint8_t* w = a.wc + (size_t)u.e * a.K * a.wb * kF8Block;
  const float* ws = a.wf + (size_t)u.e * f8_blocks(a.K) * a.wb;
  floatx4_t acc = {};
  for (int p = wave; p < a.xb; p += 4) {
    const uint4* xp = reinterpret_cast<const uint4*>(x + (size_t)p * kF8Block);
    int8v_t m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t v = 0;
#pragma unroll
      for (int z = 0; z < 4; ++z)
        v |= (uint32_t)w[(size_t)min(p * kF8Block + 32 * g + 4 * i + z, a.K - 1) * a.wb * kF8Block + n0 + r] << (8 * z);
      m[i] = (int)v;
    }
    const float s = a.xf[(size_t)row * a.xb + p] * ws[(size_t)p * a.wb + n0 / kF8Block];
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

// Rows or tiles: the rows' kernel reads the matrix again for every 16 rows and has a group's rows in one workgroup each, tiles
// take twice as long for one. So rows where there are at most two workgroups of 32 results a CU, and up to 256 rows. Measured, rows against tiles:
// one matrix [1024, 2048], 32 rows (64 workgroups) 5.1 us against 10.9, 128 (256) 7.2 against 13.6; [8192, 8192], 32 rows
// (512) 33 against 37, 64 (1,024) 68 against 42; [4096, 1024], 64 rows (512) 9.1 against 8.4, 96 (768) 12.5 against 9.5; experts
// [1024, 2048], 11 rows (352) 9.1 against 15.6, 44 (1,408) 20 against 25; [2048, 512], 5 rows (320) 8.1 against 9.9, 22
// (1,408) 18 against 12.8. The turned matrix is always on tiles, which transpose as they read; rows_back, which gathers bytes, is
// for what they cannot address.
// Not borne out by that for few rows of many groups with long rows: 2, 3 and 4 tokens that pick 10 different experts each and a
// shared one, [1024, 2048] (704, 1,056 and 1,408 workgroups), take 12.2, 15.5 and 20.1 us on rows, 17.1, 17.6 and 27.9 on the tiles that
// the rule takes (with strips of 256 the last 25.5). The rule counts workgroups, not the blocks of their contraction.
// Workgroups of 16 results, narrow, where even those leave CUs over: [4096, 1024], 16 rows (128 of 32) 4.3 us against 5.2, 32
// rows (256) 7.5 against 5.8.
hipError_t launch_f8_product(const F8Args& a, hipStream_t s) {
  const int units = a.offsets ? a.A : (a.A + kRows - 1) / kRows;
  const long long groups32 = (long long)units * ((a.N + 31) / 32);
  if ((a.back || a.A > 256 || groups32 > 2 * device_cus()) && f8_tiles_can(a)) return launch_f8_tiles(a, s);
  if (a.back) {
    const dim3 g(units, (a.N + 15) / 16);
    if (a.exact) MOE_LAUNCH("f8_rows_back", s, rows_back<true>, g, dim3(256), 0, s, a);
    else MOE_LAUNCH("f8_rows_back", s, rows_back<false>, g, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  const bool narrow = groups32 * 2 <= device_cus();
  const dim3 g(units, narrow ? (a.N + 15) / 16 : (a.N + 31) / 32);
  if (a.exact && narrow) MOE_LAUNCH("f8_rows", s, (rows_product<true, 1>), g, dim3(256), 0, s, a);
  else if (a.exact) MOE_LAUNCH("f8_rows", s, (rows_product<true, 2>), g, dim3(256), 0, s, a);
  else if (narrow) MOE_LAUNCH("f8_rows", s, (rows_product<false, 1>), g, dim3(256), 0, s, a);
  else MOE_LAUNCH("f8_rows", s, (rows_product<false, 2>), g, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
