// Quantisation of rows to microscaled 4-bit blocks, and back.
//
// A block's scale is the power of two that brings its largest magnitude into
// [4, 8): 2^(floor(log2 max) - 2), byte floor(log2 max) - 2 + 127, not below
// 0 (a block of zeros: byte 0). Magnitudes over the scale go to the nearest of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6, a tie to the even code, past 6 to 6. A NaN or an
// infinity makes its block NaN (byte 255, codes 0).
#include "mx4.h"
#include "topk.h"

namespace moe {
namespace {

// The row of piece i of n, `per` pieces a row.
__device__ inline long long piece_row(long long i, int per, long long n) {
  return n <= 0xFFFFFFFFLL ? (long long)((uint32_t)i / (uint32_t)per) : i / per;
}

// 16 bytes of values a lane, neighbours side by side: eight bf16 values and a
// dword of codes, four lanes a block, or four float32 values and half a dword,
// eight lanes a block. The block's largest magnitude by quad swaps (and a
// half-row mirror). One pass over the data; bound by memory. FLAT: rows without
// a gap and of whole blocks, one long row.
template <bool BF, bool FLAT>
__global__ __launch_bounds__(256) void quantize(const void* __restrict__ x, long long ld, int rows, int K,
                                                bool vec, uint8_t* __restrict__ codes,
                                                uint8_t* __restrict__ scales) {
  constexpr int V = BF ? 8 : 4;
  const int nb = mx4_blocks(K), per = 32 / V;  // pieces of a block
  const long long n = (long long)rows * nb * per;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = FLAT ? 0 : piece_row(i, nb * per, n);
    const int c = FLAT ? 0 : (int)(i - r * (nb * per)) * V;
    float f[V];
    if constexpr (BF) {
      const uint4 u = FLAT ? static_cast<const uint4*>(x)[i]
                           : load8_bf16(static_cast<const uint16_t*>(x) + r * ld, c, K, vec);
      f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
      f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
    } else {
      const float* p = static_cast<const float*>(x) + (FLAT ? i * V : r * ld + c);
      if (FLAT || (vec && c + V <= K)) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = c + j < K ? p[j] : 0.f;
      }
    }
    // magnitudes as integers: ordered like the floats, NaN above infinity
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    top = max(top, dpp(top, 0xB1));
    top = max(top, dpp(top, 0x4E));
    if (!BF) top = max(top, dpp(top, 0x141));
    // exponent field of max; a subnormal max has field 0, far below the least byte
    const uint32_t field = top >> 23;
    const uint32_t byte = field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
    const float sc = mx4_scale(byte);
    uint32_t w = 0;
    if (byte != 255u) {
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], sc, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], sc, 1);
      if constexpr (BF) {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], sc, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], sc, 3);
      }
    }
    if constexpr (BF) reinterpret_cast<uint32_t*>(codes)[i] = w;
    else reinterpret_cast<uint16_t*>(codes)[i] = (uint16_t)w;
    if (i % per == 0) scales[i / per] = (uint8_t)byte;
  }
}

// 16 bytes of results a lane, neighbours side by side: eight bf16 values from a
// dword of codes, or four float32 values from half of one (a lane that wrote
// the eight float32 values of its dword stored every other 16 bytes at a time:
// 191 us against 123 for 512 MiB of results).
template <bool BF, bool FLAT>
__global__ __launch_bounds__(256) void dequantize(const uint8_t* __restrict__ codes,
                                                  const uint8_t* __restrict__ scales, int rows, int K,
                                                  bool vec, void* __restrict__ y) {
  constexpr int V = BF ? 8 : 4;
  const int nb = mx4_blocks(K), per = 32 / V;  // pieces of a block
  const long long n = (long long)rows * nb * per;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = FLAT ? 0 : piece_row(i, nb * per, n);
    const int c = FLAT ? 0 : (int)(i - r * (nb * per)) * V;
    const float sc = mx4_scale(scales[i / per]);
    uint32_t p[V / 2];
    if constexpr (BF) {
      const uint4 v = __builtin_bit_cast(uint4, mx4_frag(reinterpret_cast<const uint32_t*>(codes)[i], sc));
      p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    } else {
      const uint32_t w = reinterpret_cast<const uint16_t*>(codes)[i];
      p[0] = mx4_pair<0>(w, sc);
      p[1] = mx4_pair<1>(w, sc);
    }
    if (BF) {
      uint16_t* o = static_cast<uint16_t*>(y) + (FLAT ? i * V : r * K + c);
      if (FLAT || (vec && c + V <= K)) {
        *reinterpret_cast<uint4*>(o) = make_uint4(p[0], p[1], p[V / 2 - 2], p[V / 2 - 1]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (c + j < K) o[j] = (uint16_t)(p[j / 2] >> (16 * (j & 1)));
      }
    } else {
      float* o = static_cast<float*>(y) + (FLAT ? i * V : r * K + c);
      if (FLAT || (vec && c + V <= K)) {
        *reinterpret_cast<float4*>(o) = make_float4(bf16_lo(p[0]), bf16_hi(p[0]), bf16_lo(p[1]), bf16_hi(p[1]));
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (c + j < K) o[j] = j & 1 ? bf16_hi(p[j / 2]) : bf16_lo(p[j / 2]);
      }
    }
  }
}

int grid_of(long long n) {
  const long long g = (n + 255) / 256, most = (long long)device_cus() * 32;
  return (int)(g < most ? g : most);
}

}  // namespace

hipError_t launch_mx4_quantize(const void* x, int xdtype, long long ld, int rows, int K, uint8_t* codes,
                               uint8_t* scales, hipStream_t s) {
  const dim3 g(grid_of((long long)rows * mx4_blocks(K) * (xdtype == 1 ? 4 : 8)));
  uint8_t* c = codes;
  const bool vec = rows_vec(x, ld, xdtype == 1 ? 2 : 4);
  const bool flat = vec && ld == K && K % 32 == 0;
#define QUANTIZE(BF, FLAT) \
  MOE_LAUNCH("mx4_quantize", s, (quantize<BF, FLAT>), g, dim3(256), 0, s, x, ld, rows, K, vec, c, scales)
  if (xdtype == 1) {
    if (flat) QUANTIZE(true, true);
    else QUANTIZE(true, false);
  } else {
    if (flat) QUANTIZE(false, true);
    else QUANTIZE(false, false);
  }
#undef QUANTIZE
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int K, int ydtype,
                                 void* y, hipStream_t s) {
  const dim3 g(grid_of((long long)rows * mx4_blocks(K) * (ydtype == 1 ? 4 : 8)));
  const uint8_t* c = codes;
  const bool vec = rows_vec(y, K, ydtype == 1 ? 2 : 4);
  const bool flat = vec && K % 32 == 0;
#define DEQUANTIZE(BF, FLAT) \
  MOE_LAUNCH("mx4_dequantize", s, (dequantize<BF, FLAT>), g, dim3(256), 0, s, c, scales, rows, K, vec, y)
  if (ydtype == 1) {
    if (flat) DEQUANTIZE(true, true);
    else DEQUANTIZE(true, false);
  } else {
    if (flat) DEQUANTIZE(false, true);
    else DEQUANTIZE(false, false);
  }
#undef DEQUANTIZE
  return hipGetLastError();
}

}  // namespace moe
