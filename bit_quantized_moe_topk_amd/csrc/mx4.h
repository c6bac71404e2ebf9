// Microscaled 4-bit operands: the block format and the device helpers that the
// quantisation and the products share (header-only; not part of the ABI).
//
// 32 consecutive values of a row are one block: 16 bytes of codes (two a byte,
// the first in the low half) and one scale byte s. A code is a sign bit and an
// E2M1 magnitude, one of 0, 0.5, 1, 1.5, 2, 3, 4, 6; the value is that times
// 2^(s - 127); s = 255 makes the block NaN. The gfx950 conversions take the
// scale as the exponent field of a float: byte 0 as 2^-127 and byte 255 as NaN
// (checked on the card for all 4,096 pairs of byte and code), so a scale byte
// shifted into place needs no further care. A value has at most two
// significant bits, so it is exact in bf16 as in float32 (from 2^128 on, scale
// bytes 253 and 254, it is infinite in both).
#pragma once

#include "common.h"
#include "gemv.h"

namespace moe {

typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef float floatx16_t __attribute__((ext_vector_type(16)));
typedef int int8v_t __attribute__((ext_vector_type(8)));

constexpr int kMx4 = 4;  // x type code of microscaled rows (MOE_MX4)
constexpr int kMx4MaxRows = 1 << 22;  // rows of a product

__host__ __device__ inline int mx4_blocks(int K) { return (K + 31) / 32; }

__device__ inline float mx4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Byte b of w as two values in bf16 (the first in the low half).
template <int B>
__device__ inline uint32_t mx4_pair(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
}

// The eight values of a code dword as a bf16 matrix-core operand.
__device__ inline bf16x8_t mx4_frag(uint32_t w, float scale) {
  const uint4 v = make_uint4(mx4_pair<0>(w, scale), mx4_pair<1>(w, scale), mx4_pair<2>(w, scale),
                             mx4_pair<3>(w, scale));
  return __builtin_bit_cast(bf16x8_t, v);
}

// A float32 value as the sum of three bf16 values: the top 16 bits, the top 16
// bits of what is left, and the rest (8 significant bits each), so that three
// bf16 products give the float32 product with exact weights. From 2^-110 on the
// sum is the value; smaller ones lose the bits below 2^-133, the least that bf16
// holds. What is not finite keeps its class in the first part alone. An infinite
// weight (from 2^128 on) makes NaN with lower parts that are zero. Cutting it to
// a finite one for them took 3 to 14 % of a float32 product's time (64 tokens x
// 11, 512 experts, [2048, 512]: 58 us against 53, its gradient 106 against 93),
// a path of its own past a branch up to 25 %: left out, as quantisation never
// writes such scale bytes (253, 254).
struct Split3 {
  uint32_t h, m, l;  // bf16 bits in the high half
};
__device__ inline Split3 split3(float v) {
  Split3 s;
  const uint32_t u = __float_as_uint(v);
  const bool fin = (u & 0x7F800000u) != 0x7F800000u;
  s.h = u & 0xFFFF0000u;
  if (!fin && (u & 0x007FFFFFu)) s.h |= 0x00400000u;  // NaN stays NaN without its low bits
  const float r = fin ? v - __uint_as_float(s.h) : 0.f;
  s.m = __float_as_uint(r) & 0xFFFF0000u;
  s.l = __float_as_uint(r - __uint_as_float(s.m));
  return s;
}

__device__ inline uint32_t hi_pair(uint32_t a, uint32_t b) {  // high halves of a (low) and b (high)
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ inline uint32_t lo_pair(uint32_t a, uint32_t b) {  // low halves
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

// Eight float32 values as three bf16 operands.
__device__ inline void split3x8(const float (&f)[8], uint4& h, uint4& m, uint4& l) {
  Split3 s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = split3(f[i]);
  h = make_uint4(hi_pair(s[0].h, s[1].h), hi_pair(s[2].h, s[3].h), hi_pair(s[4].h, s[5].h), hi_pair(s[6].h, s[7].h));
  m = make_uint4(hi_pair(s[0].m, s[1].m), hi_pair(s[2].m, s[3].m), hi_pair(s[4].m, s[5].m), hi_pair(s[6].m, s[7].m));
  l = make_uint4(hi_pair(s[0].l, s[1].l), hi_pair(s[2].l, s[3].l), hi_pair(s[4].l, s[5].l), hi_pair(s[6].l, s[7].l));
}

// One product launch. Rows s in [0, A) lie in the groups that `offsets`
// describes (group e: rows offsets[e] .. offsets[e + 1], matrix e), or all
// belong to the one matrix (offsets null). perm not null: row s reads x's row
// token_of(perm[s], T, k).
struct Mx4Args {
  const void* x;          // rows of float32, bf16 or codes
  const uint8_t* xs;      // scales of x's rows (kMx4)
  int xdtype;
  long long ldx;          // elements between x's rows (float32, bf16)
  int A, T, k, E_tot;
  const int32_t* offsets;
  const int32_t* perm;
  const uint8_t* wc;      // [E_tot][N][16 blocks]
  const uint8_t* ws;      // [E_tot][N][blocks]
  int N, K;
  void* y;                // [A][N] (forward), [A][K] (gradient)
  int ydtype;
  uint32_t* counter;      // of the tiles taken, or null: tiles are dealt in turn
};

// About how many 128-row tiles the rows make: a group that has rows has one at least.
inline long long mx4_row_tiles(const Mx4Args& a) {
  const long long full = ((long long)a.A + 127) / 128, groups = a.A < a.E_tot ? a.A : a.E_tot;
  return full > groups ? full : groups;
}

// The token of an assignment id, -1 of one outside [0, A) (asked of the id: those from -(k - 1) to -1 divided by k
// are 0).
__device__ inline int mx4_token(const Mx4Args& a, int id) {
  return (unsigned)id < (unsigned)a.A ? token_of(id, a.T, a.k) : -1;
}

// x's row that row s of the groups reads; -1: none (an id out of range).
__device__ inline int mx4_row(const Mx4Args& a, int s) { return a.perm ? mx4_token(a, a.perm[s]) : s; }

// An offset cut to the rows, and so the first row of group e.
__device__ inline int cut_offset(const Mx4Args& a, int offset) { return min(max(offset, 0), a.A); }
__device__ inline int first_row(const Mx4Args& a, int e) { return cut_offset(a, a.offsets[e]); }

// The group of row s: how many of offsets[1 .. E_tot] are at most s (one wave,
// every lane gets it; 512 offsets on their way at once). E_tot: the row is
// behind the last group.
__device__ inline int mx4_group_of(const int32_t* __restrict__ offsets, int E_tot, int s) {
  const int lane = threadIdx.x & 63;
  int e = 0;
  for (int b = 0; b < E_tot; b += 512) {
    int v[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) v[z] = offsets[min(b + 64 * z + lane, E_tot - 1) + 1];
#pragma unroll
    for (int z = 0; z < 8; ++z) e += __popcll(__ballot(b + 64 * z + lane < E_tot && v[z] <= s));
  }
  return e;
}

// Eight consecutive values from column c of a row of n (zeros past n), as
// float32 values or as bf16 bits. vec: the row is 16-byte aligned.
__device__ inline uint4 load8_bf16(const uint16_t* __restrict__ row, int c, int n, bool vec) {
  if (vec && c + 8 <= n) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c + i < n ? row[c + i] : 0u;
  return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}
__device__ inline void load8_f32(const float* __restrict__ row, int c, int n, bool vec, float (&f)[8]) {
  if (vec && c + 8 <= n) {
    const float4 p = *reinterpret_cast<const float4*>(row + c), q = *reinterpret_cast<const float4*>(row + c + 4);
    f[0] = p.x; f[1] = p.y; f[2] = p.z; f[3] = p.w;
    f[4] = q.x; f[5] = q.y; f[6] = q.z; f[7] = q.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = c + i < n ? row[c + i] : 0.f;
}

// Whether rows `ld` elements of `size` bytes apart can be read 16 bytes at a time.
inline bool rows_vec(const void* p, long long ld, int size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * size) % 16 == 0;
}

// ---- launchers (each returns hipGetLastError() after enqueueing) ----------
hipError_t launch_mx4_quantize(const void* x, int xdtype, long long ld, int rows, int K, uint8_t* codes,
                               uint8_t* scales, hipStream_t s);
hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int K, int ydtype,
                                 void* y, hipStream_t s);
hipError_t launch_mx4_forward(const Mx4Args& a, hipStream_t s);
hipError_t launch_mx4_gradient(const Mx4Args& a, hipStream_t s);
hipError_t launch_mx4_tiles(Mx4Args a, hipStream_t s);
void launch_mx4_zero(uint32_t* counter, hipStream_t s);
hipError_t launch_mx4_grad_tiles(Mx4Args a, hipStream_t s);
hipError_t launch_mx4_few(const Mx4Args& a, hipStream_t s);
bool mx4_tiles4_can(const Mx4Args& a);
hipError_t launch_mx4_tiles4(Mx4Args a, hipStream_t s);
hipError_t launch_mx4_sum_tokens(const float* part, const int32_t* slot_of, const int32_t* offsets, int E_tot, int T,
                                 int k, int has_shared, int A, int K, void* y, int ydtype, hipStream_t s);

}  // namespace moe
