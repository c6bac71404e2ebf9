// Products of few rows with a microscaled matrix: y[s][n] = sum_k x[row(s)][k]
// W[e(s)][n][k], and the gradient dx[s][k] = sum_n dy[s][n] W[e(s)][n][k].
//
// Up to 16 rows of one group and a strip of the matrix per workgroup, on
// 16x16 matrix-core tiles. Weights go from memory to registers, where they
// become bf16 exactly; float32 rows enter as three exact bf16 parts, so that
// every product is exact and only the float32 sums round. Bound by the
// matrix's bytes: each is read once per 16 rows.
#include "mx4_tile.h"

namespace moe {
namespace {

constexpr int kRows = 16;   // rows of a group per workgroup
constexpr int kCols = 128;  // matrix columns per workgroup (gradient)

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

__device__ inline void store_out(const Mx4Args& a, size_t i, float v) {
  if (a.ydtype == 1) static_cast<uint16_t*>(a.y)[i] = (uint16_t)f32_to_bf16_bits(v);
  else static_cast<float*>(a.y)[i] = v;
}

// Four waves share K in whole chunks of 128: lane (r, g) holds block g of a chunk of
// matrix row r (its 16 bytes of codes, one scale) and of x's row r. A product
// step takes eight values of each of the four blocks; the order of K within a
// chunk is the same for both operands, which is all that matters. Microscaled
// rows go through the 4-bit matrix cores, one product a chunk. A wave asks for
// several chunks at once: with a few rows the time is the chain from the
// group's offsets over its loads to the sums.
template <int XT, int NT>
__global__ __launch_bounds__(256) void rows_forward(Mx4Args a, bool vec) {
  constexpr int kAhead = XT == 0 ? 2 : 4;  // chunks on their way at once, of weights and rows
  __shared__ float part[4][NT][kRows * 16];
  const Unit u = unit_of(a);
  if (u.M <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  const int nb = mx4_blocks(a.K), n0 = blockIdx.y * 16 * NT;
  const uint4* wc[NT];
  const uint8_t* ws[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const size_t row = (size_t)u.e * a.N + min(n0 + 16 * j + r, a.N - 1);
    wc[j] = reinterpret_cast<const uint4*>(a.wc) + row * nb;
    ws[j] = a.ws + row * nb;
  }
  const int xr = r < u.M ? mx4_row(a, u.s0 + r) : -1;
  floatx4_t acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = floatx4_t{};
  const int share = 4 * ((nb + 15) / 16), end = min(nb, share * (wave + 1));  // blocks of a wave, whole chunks
  for (int b0 = share * wave; b0 < end; b0 += 4 * kAhead) {
    uint4 c[kAhead][NT];
    uint32_t sw[kAhead][NT];
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      const int b = b0 + 4 * z + g;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        c[z][j] = make_uint4(0, 0, 0, 0);
        sw[z][j] = 0;
        if (b < end) {
          c[z][j] = wc[j][b];
          sw[z][j] = ws[j][b];
        }
      }
    }
    if constexpr (XT == kMx4) {
      uint4 xc[kAhead];
      uint32_t sx[kAhead];
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        const int b = b0 + 4 * z + g;
        xc[z] = make_uint4(0, 0, 0, 0);
        sx[z] = 0;
        if (b < end && xr >= 0) {
          xc[z] = reinterpret_cast<const uint4*>(a.x)[(size_t)xr * nb + b];
          sx[z] = a.xs[(size_t)xr * nb + b];
        }
      }
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        if (b0 + 4 * z >= end) break;
        const int8v_t B = {(int)xc[z].x, (int)xc[z].y, (int)xc[z].z, (int)xc[z].w, 0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 w = c[z][j];
          const int8v_t A = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
          acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc[j], 4, 4, 0, (int)sw[z][j], 0, (int)sx[z]);
        }
      }
    } else {
      uint4 x1[XT == 1 ? kAhead : 1][4];
      float x3[XT == 0 ? kAhead : 1][4][8];
#pragma unroll
      for (int z = 0; z < kAhead; ++z)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int b = b0 + 4 * z + g, k = 32 * b + 8 * i;
          const bool there = xr >= 0 && b < end && k < a.K;
          if constexpr (XT == 1) {
            x1[z][i] = make_uint4(0, 0, 0, 0);
            if (there) x1[z][i] = load8_bf16(static_cast<const uint16_t*>(a.x) + xr * a.ldx, k, a.K, vec);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x3[z][i][e] = 0.f;
            if (there) load8_f32(static_cast<const float*>(a.x) + xr * a.ldx, k, a.K, vec, x3[z][i]);
          }
        }
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        if (b0 + 4 * z >= end) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 v[XT == 1 ? 1 : 3];
          if constexpr (XT == 1) v[0] = x1[z][i];
          else split3x8(x3[z][i], v[0], v[1], v[2]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 w = c[z][j];
            const bf16x8_t wf = mx4_frag(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w, mx4_scale(sw[z][j]));
#pragma unroll
            for (int p = XT == 1 ? 0 : 2; p >= 0; --p)
              acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8_t, v[p]), acc[j], 0, 0, 0);
          }
        }
      }
    }
  }
  // acc[j][i]: matrix row 16 j + 4 g + i, x's row r
#pragma unroll
  for (int j = 0; j < NT; ++j)
    *reinterpret_cast<floatx4_t*>(&part[wave][j][16 * r + 4 * g]) = acc[j];
  __syncthreads();
  for (int i = tid; i < 256 * NT; i += 256) {
    const int m = (i / (16 * NT)), n = i % (16 * NT), at = 16 * m + n % 16;
    if (m < u.M && n0 + n < a.N)
      store_out(a, (size_t)(u.s0 + m) * a.N + n0 + n,
                (part[0][n / 16][at] + part[1][n / 16][at]) + (part[2][n / 16][at] + part[3][n / 16][at]));
  }
}

// Four waves share N in steps of 32. Lane (r, g) holds, for each of the eight
// matrix rows n = 8 g + j of a step, one dword of codes: columns k0 + 8 r ..
// + 7. Converted row by row (one scale each) the values pair up along k; two
// rows' pairs are then regrouped along n, so that eight conversions' worth of
// registers give the operands of eight 16x16x32 products, product c covering
// columns k0 + 8 r + c. No transposed copy of the matrix is needed.
// The next step's are on their way while one is used: every load is issued in
// any case, within the matrix and the rows, and what lies past N counts as zeros
// (a way past the loads would have the products wait for them).
template <int DT>
struct GradRegs {
  uint32_t w[8], s[8];
  uint4 d[DT == 1 ? 1 : 2];
};
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void rows_gradient(Mx4Args a) {
  __shared__ float part[4][kRows * kCols];
  const Unit u = unit_of(a);
  if (u.M <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  const int nb = mx4_blocks(a.K), k0 = blockIdx.y * kCols;
  const int piece = min(k0 / 8 + r, 4 * nb - 1);  // dword of codes in a matrix row (past it: not stored)
  const uint32_t* wc = reinterpret_cast<const uint32_t*>(a.wc) + (size_t)u.e * a.N * nb * 4 + piece;
  const uint8_t* ws = a.ws + (size_t)u.e * a.N * nb + piece / 4;
  const char* row = static_cast<const char*>(a.x) + (size_t)(u.s0 + min(r, u.M - 1)) * a.ldx * (DT == 1 ? 2 : 4);
  auto load = [&](int n0, GradRegs<DT>& v) __attribute__((always_inline)) {
    const int n = n0 + 8 * g;
    if constexpr (VEC) {
      const uint4* p = reinterpret_cast<const uint4*>(row + (size_t)min(n, a.N - 8) * (DT == 1 ? 2 : 4));
      v.d[0] = p[0];
      if constexpr (DT != 1) v.d[1] = p[1];
    } else if (n < a.N) {
      if constexpr (DT == 1) {
        v.d[0] = load8_bf16(reinterpret_cast<const uint16_t*>(row), n, a.N, false);
      } else {
        float f[8];
        load8_f32(reinterpret_cast<const float*>(row), n, a.N, false, f);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v.d[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                              __float_as_uint(f[4 * i + 3]));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const size_t at = (size_t)min(n + j, a.N - 1) * nb;
      v.w[j] = wc[4 * at];
      v.s[j] = ws[at];
    }
  };
  floatx4_t acc[8] = {};
  auto step = [&](int n0, const GradRegs<DT>& v, GradRegs<DT>& next) __attribute__((always_inline)) {
    load(n0 + 128, next);
    __builtin_amdgcn_sched_barrier(0);
    const int n = n0 + 8 * g;
    uint32_t p[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sc = mx4_scale(n + j < a.N ? v.s[j] : 0u);
      p[j][0] = mx4_pair<0>(v.w[j], sc);
      p[j][1] = mx4_pair<1>(v.w[j], sc);
      p[j][2] = mx4_pair<2>(v.w[j], sc);
      p[j][3] = mx4_pair<3>(v.w[j], sc);
    }
    uint4 d[3], x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = n < a.N ? v.d[DT == 1 ? 0 : i] : make_uint4(0, 0, 0, 0);
    if constexpr (DT == 1) {
      d[0] = x[0];
    } else {
      const float f[8] = {__uint_as_float(x[0].x), __uint_as_float(x[0].y), __uint_as_float(x[0].z), __uint_as_float(x[0].w),
                          __uint_as_float(x[1].x), __uint_as_float(x[1].y), __uint_as_float(x[1].z), __uint_as_float(x[1].w)};
      split3x8(f, d[0], d[1], d[2]);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      auto two = [&](int j) {
        return c & 1 ? hi_pair(p[j][c / 2], p[j + 1][c / 2]) : lo_pair(p[j][c / 2], p[j + 1][c / 2]);
      };
      const bf16x8_t wf = __builtin_bit_cast(bf16x8_t, make_uint4(two(0), two(2), two(4), two(6)));
#pragma unroll
      for (int q = DT == 1 ? 0 : 2; q >= 0; --q)
        acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, d[q]), wf, acc[c], 0, 0, 0);
    }
  };
  GradRegs<DT> even, odd;
  load(32 * wave, even);
  for (int n0 = 32 * wave; n0 < a.N; n0 += 256) {
    step(n0, even, odd);
    if (n0 + 128 < a.N) step(n0 + 128, odd, even);
  }
  // acc[c][i]: row 4 g + i, column k0 + 8 r + c
#pragma unroll
  for (int c = 0; c < 8; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][(4 * g + i) * kCols + 8 * r + c] = acc[c][i];
  __syncthreads();
  for (int i = tid; i < u.M * kCols; i += 256) {
    const int k = k0 + i % kCols;
    if (k < a.K)
      store_out(a, (size_t)(u.s0 + i / kCols) * a.K + k, (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]));
  }
}

// dx[t] = the sum of a token's rows of part, in the order of its assignments
// (the shared expert's last); float32 sums, one rounding. Rows of part that are in
// no group were not written and add nothing. A lane adds up four columns (where K
// is no multiple of four, one), four rows on their way at once.
template <bool BF, int V>
__global__ __launch_bounds__(256) void sum_tokens(const float* __restrict__ part, const int32_t* __restrict__ slot_of,
                                                  const int32_t* __restrict__ offsets, int E_tot, int T, int k,
                                                  int has_shared, int A, int K, void* __restrict__ y) {
  const int t = blockIdx.x, n = k + has_shared, lo = max(offsets[0], 0), hi = min(offsets[E_tot], A);
  for (int c = V * (blockIdx.y * 256 + threadIdx.x); c < K; c += V * gridDim.y * 256) {
    float v[V] = {};
    for (int j0 = 0; j0 < n; j0 += 4) {
      float p[4][V];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int j = j0 + z;
        const int s = j < n ? slot_of[j < k ? (size_t)t * k + j : (size_t)T * k + t] : -1;
#pragma unroll
        for (int i = 0; i < V; ++i) p[z][i] = 0.f;
        if (s >= lo && s < hi) {
          if constexpr (V == 4) {
            const float4 q = *reinterpret_cast<const float4*>(part + (size_t)s * K + c);
            p[z][0] = q.x; p[z][1] = q.y; p[z][2] = q.z; p[z][3] = q.w;
          } else {
            p[z][0] = part[(size_t)s * K + c];
          }
        }
      }
#pragma unroll
      for (int z = 0; z < 4; ++z)
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += p[z][i];
    }
    const size_t at = (size_t)t * K + c;
    if constexpr (V == 4) {
      if (BF)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) =
            make_uint2(f32_to_bf16_bits(v[0]) | f32_to_bf16_bits(v[1]) << 16,
                       f32_to_bf16_bits(v[2]) | f32_to_bf16_bits(v[3]) << 16);
      else
        *reinterpret_cast<float4*>(static_cast<float*>(y) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      if (BF) static_cast<uint16_t*>(y)[at] = (uint16_t)f32_to_bf16_bits(v[0]);
      else static_cast<float*>(y)[at] = v[0];
    }
  }
}

// Which kernels take a product of these rows. Times: us a call in a chain of
// calls; experts: 512 and a shared one, 10 a token, evenly loaded, or with a few
// popular ones (a load that falls with the rank as 1 / rank^1.1).
//
// kFewRows (a workgroup for 16 rows and a strip of the matrix, all of them in
// one launch) is the quickest to begin: up to 32 rows in groups (2 tokens x 11
// bf16, [1024, 2048]: 12 against kFew's 14 and the tiles' 15), and for one matrix
// until the 16-row units fill the chip a few times over (bf16, [1024, 2048]: 256
// rows 10 against the tiles' 17, 512 rows 18 against 17, 1,024 rows 32 against
// 17; 4-bit rows: 14 against 15 for 512, 25 against 16 for 1,024).
// kFew (the same 16 rows, from one list of all groups' tiles, the matrix read
// ahead) reads each matrix once where groups hold a handful of rows. Float32
// rows, whose parts it makes once for all waves: up to 80 rows a group ([2048,
// 512], against the tiles: 64 tokens 55 / 163, with popular experts 19 / 37;
// 2,000 tokens 240 / 319; 3,500: 388 / 398; 5,000: 542 / 518; 16 experts,
// [1024, 2048]: 100 rows a group 41 / 91, 384 rows 119 / 98), and for one matrix
// from half a tile for every CU up to four ([1024, 2048], kFewRows, kFew, tiles:
// 256 rows 17, 23, 89; 1,024 rows 51, 26, 89; 8,192 rows 410, 142, 105). bf16
// rows: up to 12 a group ([2048, 512]: 256 tokens 68 / 90, 1,024 tokens 121 /
// 110), with more than 1,024 columns up to 3 ([1024, 2048], popular experts: 32
// tokens 23 / 31, evenly loaded 74 / 64; 256 tokens 71 / 57, evenly 164 / 147),
// and there only with four strips for every CU, as one wave goes through all
// columns (4 tokens 14.6 / 15.0).
// kTiles: the rest. Grouped 4-bit rows from 32 on (against kFewRows; [1024,
// 2048]: 4 tokens 15 / 18, 16 tokens 38 / 52, 64 tokens 84 / 167, where reading
// the matrices takes 80; [2048, 512]: 13 / 11, 29 / 34, 58 / 109).
enum Kernels { kFewRows, kFew, kTiles };

Kernels forward_kernels(const Mx4Args& a) {
  const long long cus = device_cus(), units = (a.A + kRows - 1) / kRows, strips = (a.N + 255) / 256;
  if (!a.offsets) {
    if (a.xdtype != 0) return units * ((a.N + 31) / 32) > 4 * cus ? kTiles : kFewRows;
    return 2 * units * strips < cus ? kFewRows : units * strips <= 4 * cus ? kFew : kTiles;
  }
  if (a.A < 32) return kFewRows;
  if (a.xdtype == kMx4) return kTiles;
  if (a.xdtype == 0) return a.A <= (long long)kFewRowsF32 * a.E_tot ? kFew : kTiles;
  const bool deep = a.K > 1024;
  const long long groups = a.A < a.E_tot ? a.A : a.E_tot;
  return a.A <= (deep ? 3LL : 12LL) * a.E_tot && 2 * groups * strips >= (deep ? 4 : 1) * cus ? kFew : kTiles;
}

// Gradients: tiles where groups hold more than a few rows and there are more than 256 (tiles against 16-row units, as
// above). bf16 rows from 4 a group on ([2048, 512]: 64 tokens 72 / 67, 256 tokens 99 / 119, 400 tokens 95 / 139; [1000,
// 2048], which is not streamed: 64 tokens 243 / 166, 256 tokens 347 / 277, with popular experts 103 / 210; 17 experts,
// [1024, 2048]: 192 rows 21 / 22, 500 rows 25 / 28). Float32 rows from 12 ([2048, 512]: 256 tokens 501 / 168, 1,000 tokens
// 555 / 406, 2,000 tokens 746 / 790; 17 experts, [1000, 2048]: 16 rows a group 45 / 57, 45 rows 66 / 49, 64 rows 80 / 156: by
// how the rows fall on tiles, either leads from 12 to 45 a group). One matrix, [1024, 2048]: from about eight 16-row units
// for every CU on (bf16: 2,048 rows 35 / 32, 4,096 rows 36 / 57; float32: 4,096 rows 99 / 93).
bool gradient_tiles_pay(const Mx4Args& a) {
  const bool f32 = a.xdtype == 0;
  if (a.offsets) return a.A > (f32 ? 12LL : 4LL) * a.E_tot && a.A > 256;
  const long long units = (a.A + kRows - 1) / kRows;
  return units * ((a.K + kCols - 1) / kCols) > (f32 ? 10 : 8) * device_cus();
}

__global__ __launch_bounds__(256) void zero_counters(uint32_t* p) { p[threadIdx.x] = 0u; }

}  // namespace

void launch_mx4_zero(uint32_t* counter, hipStream_t s) {
  MOE_LAUNCH("mx4_zero", s, zero_counters, dim3(1), dim3(256), 0, s, counter);
}

hipError_t launch_mx4_forward(const Mx4Args& a, hipStream_t s) {
  const Kernels take = forward_kernels(a);
  if (take == kFew) return launch_mx4_few(a, s);
  if (take == kTiles) {
    if (a.xdtype != kMx4) return launch_mx4_tiles(a, s);
    if (mx4_tiles4_can(a)) return launch_mx4_tiles4(a, s);
  }
  const bool vec = a.xdtype != kMx4 && rows_vec(a.x, a.ldx, a.xdtype == 1 ? 2 : 4);
  // 32 matrix rows a workgroup, or 16 where that leaves half of the CUs without one (one row, [1024, 2048]: bf16 4.1 us
  // against 5.8, float32 7.3 against 8.9, 4 bits 3.7 against 4.7)
  const int units = a.offsets ? a.A : (a.A + kRows - 1) / kRows;
  const bool narrow = (long long)units * ((a.N + 31) / 32) * 2 <= device_cus();
  const dim3 g(units, narrow ? (a.N + 15) / 16 : (a.N + 31) / 32);
#define ROWS(XT) \
  if (narrow) MOE_LAUNCH("mx4_rows", s, (rows_forward<XT, 1>), g, dim3(256), 0, s, a, vec); \
  else MOE_LAUNCH("mx4_rows", s, (rows_forward<XT, 2>), g, dim3(256), 0, s, a, vec)
  if (a.xdtype == kMx4) { ROWS(kMx4); }
  else if (a.xdtype == 1) { ROWS(1); }
  else { ROWS(0); }
#undef ROWS
  return hipGetLastError();
}

hipError_t launch_mx4_gradient(const Mx4Args& a, hipStream_t s) {
  if (gradient_tiles_pay(a)) return launch_mx4_grad_tiles(a, s);
  const dim3 g(a.offsets ? a.A : (a.A + kRows - 1) / kRows, (a.K + kCols - 1) / kCols);
  const bool vec = a.N % 8 == 0 && rows_vec(a.x, a.ldx, a.xdtype == 1 ? 2 : 4);
  if (a.xdtype == 1 && vec) MOE_LAUNCH("mx4_rows_grad", s, (rows_gradient<1, true>), g, dim3(256), 0, s, a);
  else if (a.xdtype == 1) MOE_LAUNCH("mx4_rows_grad", s, (rows_gradient<1, false>), g, dim3(256), 0, s, a);
  else if (vec) MOE_LAUNCH("mx4_rows_grad", s, (rows_gradient<0, true>), g, dim3(256), 0, s, a);
  else MOE_LAUNCH("mx4_rows_grad", s, (rows_gradient<0, false>), g, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_mx4_sum_tokens(const float* part, const int32_t* slot_of, const int32_t* offsets, int E_tot, int T,
                                 int k, int has_shared, int A, int K, void* y, int ydtype, hipStream_t s) {
  const bool four = K % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
  const dim3 g(T, four ? (K + 1023) / 1024 : (K + 255) / 256);
#define SUM_TOKENS(BF, V) \
  MOE_LAUNCH("mx4_sum_tokens", s, (sum_tokens<BF, V>), g, dim3(256), 0, s, part, slot_of, offsets, E_tot, T, k, \
             has_shared, A, K, y)
  if (ydtype == 1) {
    if (four) SUM_TOKENS(true, 4);
    else SUM_TOKENS(true, 1);
  } else {
    if (four) SUM_TOKENS(false, 4);
    else SUM_TOKENS(false, 1);
  }
#undef SUM_TOKENS
  return hipGetLastError();
}

}  // namespace moe
