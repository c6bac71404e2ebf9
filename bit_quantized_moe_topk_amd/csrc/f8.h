// 8-bit operands: the block format and the device helpers that the quantiser,
// the norm and the products share (header-only; not part of the ABI).
//
// A row's values are E4M3 codes, 128 of them to a block with one float32 scale
// (a row), or 128 x 128 (a matrix); rows of codes are filled up to whole blocks
// with zeros, so that every row starts on 128 bytes and no kernel looks at the end
// of a contraction.
//
// scale = max(largest magnitude, 2^-116) / 448, which is a normal number, and
// code = the exact quotient rounded once. A quotient rounded to float32 first may
// come to lie on the border between two codes (one in 1,000 values of a bf16
// row does, whose magnitudes and largest magnitude are short), so the sign of
// the exact remainder decides there (f8_quotient).
//
// The 8-bit matrix cores add up the 128 products of a 16x16x128 instruction with
// about 13 bits under the binade of the largest (65536 + 8 is kept, 65536 + 4 is
// not: measured, the same for every 8-bit form): each product may lose less than
// 2^-12 of the block's largest, all of them together 2^-5 of it, and where large
// ones cancel the small ones may be gone. Results in bf16 take them all the same: of
// normal values a row is off by 2.2e-4 of its norm, against 1.66e-3 by the result's own
// rounding (1.65892e-3 together, 1.65887e-3 with exact sums: 8,192 x 1024 x 2048), and
// a code's rounding is up to 2^-4 of each product. Exact sums, with float32 results,
// took 46 us against 25 there, 508 against 318 for the experts chunk of 8,192 tokens,
// 249 against 228 for the gradient of 1,024. Results in float32 have them, on the bf16 matrix
// cores: a code has four significant bits, so it is exact in bf16, products are
// exact, and sums keep float32's bits. Block sums are scaled and added up in
// float32 either way.
#pragma once

#include "mx4_tile.h"
#include "topk.h"

namespace moe {

constexpr int kF8Block = 128;
constexpr float kF8Least = 0x1p-116f;  // least magnitude that a scale goes by

__host__ __device__ inline int f8_blocks(int K) { return (K + kF8Block - 1) / kF8Block; }

// One product launch: y[s][n] = sum over c of x[row(s)][c] M[e(s)][n][c], N results a row and
// K columns c. Mx4Args' x and wc are codes; forward: the stored matrix is M ([N][wb 128]);
// back: it is M turned ([K][wb 128]).
struct F8Args : Mx4Args {
  const float* xf;  // [rows][xb]
  const float* wf;  // [E_tot][..][wb]
  int xb, wb;       // blocks of a row of x (along K) and of a stored row of the matrix
  bool back;
  bool exact;       // products on the bf16 matrix cores (results that stay in float32)
};

// The scale of a block whose largest magnitude is `top`.
__device__ inline float f8_scale_of(float top) { return fmaxf(top, kF8Least) / 448.f; }

// A float32 number that rounds to the code that the exact quotient of v by s rounds to. Two steps bring |v| * inv to within
// one unit of it; the sign of the exact remainder says on which side it lies. A border between two codes has an even last bit, so
// an odd number is on its own side of all of them, and an even one goes one unit towards the quotient (nine instructions in all).
__device__ inline float f8_quotient(float v, float s, float inv) {
  const float m = fabsf(v);
  float q = m * inv;
  q = fmaf(fmaf(-q, s, m), inv, q);
  const int r = __float_as_int(fmaf(-q, s, m)), u = __float_as_int(q);
  const int towards = max(min(r, 1), -1);  // -1, 0, 1 as the remainder's sign (a zero is +0)
  const float c = __int_as_float(u + (towards & ((u & 1) - 1)));
  return __builtin_copysignf(c, v);  // (a zero keeps its sign)
}

// The codes of eight values of a block whose largest magnitude is `top` (bits, ordered as
// integers): two dwords. *scale is the block's. Blocks below 2^-40 are brought up first, so that no
// remainder is lost below float32's range.
__device__ inline uint2 f8_codes(const float (&f)[8], uint32_t top, float* scale) {
  if (top >= 0x7F800000u) {
    *scale = __uint_as_float(0x7FC00000u);
    return make_uint2(0u, 0u);
  }
  float s = f8_scale_of(__uint_as_float(top)), q[8];
  *scale = s;
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = f[i];
  if (top < 0x2B800000u) {
    s *= 0x1p80f;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] *= 0x1p80f;
  }
  const float inv = 1.f / s;
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = f8_quotient(q[i], s, inv);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

__device__ inline uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The largest of eight magnitudes over the 16 lanes of a row of lanes, which hold one block.
__device__ inline uint32_t f8_top16(const float (&f)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, magnitude(f[i]));
  top = max(top, dpp(top, 0xB1));
  top = max(top, dpp(top, 0x4E));
  top = max(top, dpp(top, 0x141));
  return max(top, dpp(top, 0x140));
}

// Sixteen bytes at any element's address (global memory takes them there; a line more at times is all that it costs:
// [6853, 512] x [1330, 512] 44.7 us by elements, 19.9 so).
typedef uint32_t any16_t __attribute__((ext_vector_type(4), aligned(2)));
typedef float any16f_t __attribute__((ext_vector_type(4), aligned(4)));

// Eight values from column c of a row of n in either type (zeros past n).
template <bool BF>
__device__ inline void load8(const void* __restrict__ row, int c, int n, float (&f)[8]) {
  if constexpr (BF) {
    const uint16_t* x = static_cast<const uint16_t*>(row) + c;
    if (c + 8 <= n) {
      const any16_t u = *reinterpret_cast<const any16_t*>(x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(u[i]);
        f[2 * i + 1] = bf16_hi(u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = c + i < n ? bf16_lo(x[i]) : 0.f;
    }
  } else {
    const float* x = static_cast<const float*>(row) + c;
    if (c + 8 <= n) {
      const any16f_t a = *reinterpret_cast<const any16f_t*>(x), b = *reinterpret_cast<const any16f_t*>(x + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = a[i];
        f[4 + i] = b[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = c + i < n ? x[i] : 0.f;
    }
  }
}

// Eight values in bf16, from column c of a row of n on.
__device__ inline void store8_bf16(uint16_t* y, int c, int n, uint32_t a, uint32_t b, uint32_t d, uint32_t e) {
  const any16_t p = {a, b, d, e};
  if (c + 8 <= n) {
    *reinterpret_cast<any16_t*>(y + c) = p;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) y[c + i] = (uint16_t)(p[i / 2] >> (16 * (i & 1)));
  }
}
__device__ inline void store4_f32(float* y, int c, int n, float a, float b, float d, float e) {
  const any16f_t p = {a, b, d, e};
  if (c + 4 <= n) {
    *reinterpret_cast<any16f_t*>(y + c) = p;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < n) y[c + i] = p[i];
  }
}

template <bool BF>
__device__ inline void store8(void* __restrict__ row, int c, int n, const float (&f)[8]) {
  if constexpr (BF) {
    store8_bf16(static_cast<uint16_t*>(row), c, n, pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  } else {
    store4_f32(static_cast<float*>(row), c, n, f[0], f[1], f[2], f[3]);
    store4_f32(static_cast<float*>(row), c + 4, n, f[4], f[5], f[6], f[7]);
  }
}

// Eight codes as bf16 values, exactly.
__device__ inline bf16x8_t f8_bf16(int lo, int hi) {
  typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
  const uint4 v = make_uint4(__builtin_bit_cast(uint32_t, (pair_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false)),
                             __builtin_bit_cast(uint32_t, (pair_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true)),
                             __builtin_bit_cast(uint32_t, (pair_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false)),
                             __builtin_bit_cast(uint32_t, (pair_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true)));
  return __builtin_bit_cast(bf16x8_t, v);
}

// The 128 products of a block, 16 matrix rows (a) by 16 rows (b): lane l has 32 codes of row l % 16 of
// each; result i is matrix row 4 (l / 16) + i, row l % 16.
template <bool EXACT>
__device__ inline floatx4_t f8_products(const int8v_t& a, const int8v_t& b) {
  if constexpr (EXACT) {
    floatx4_t c = {};
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f8_bf16(a[i], a[i + 1]), f8_bf16(b[i], b[i + 1]), c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, floatx4_t{}, 0, 0, 0, 0, 0, 0);
  }
}

__device__ inline int8v_t f8_pair(uint4 a, uint4 b) {
  return int8v_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// ---- launchers (each returns hipGetLastError() after enqueueing) ----------
hipError_t launch_f8_quantize(const void* x, int xdtype, long long ld, int mats, int rows, int K, int block_rows,
                              uint8_t* codes, float* scales, hipStream_t s);
hipError_t launch_f8_dequantize(const uint8_t* codes, const float* scales, int mats, int rows, int K, int block_rows,
                                int ydtype, void* y, hipStream_t s);
hipError_t launch_f8_product(const F8Args& a, hipStream_t s);
bool f8_tiles_can(const F8Args& a);
hipError_t launch_f8_tiles(F8Args a, hipStream_t s);

}  // namespace moe
