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

// Four lanes a block, eight values a lane: the block's largest magnitude by
// two quad swaps, one dword of codes a lane (a wave writes 256 contiguous
// bytes of codes and 16 of scales). One pass over the data; bound by memory.
template <bool BF>
__global__ __launch_bounds__(256) void quantize(const void* __restrict__ x, long long ld, int rows, int K,
                                                bool vec, uint32_t* __restrict__ codes,
                                                uint8_t* __restrict__ scales) {
  const int nb = mx4_blocks(K);
  const long long n = (long long)rows * nb * 4;  // eights
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = i / (nb * 4);
    const int c = (int)(i - r * (nb * 4)) * 8;
    float f[8];
    if (BF) {
      const uint4 u = load8_bf16(static_cast<const uint16_t*>(x) + r * ld, c, K, vec);
      f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
      f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
    } else {
      load8_f32(static_cast<const float*>(x) + r * ld, c, K, vec, f);
    }
    // magnitudes as integers: ordered like the floats, NaN above infinity
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    top = max(top, dpp(top, 0xB1));
    top = max(top, dpp(top, 0x4E));
    // exponent field of max; a subnormal max has field 0, far below the least byte
    const uint32_t field = top >> 23;
    const uint32_t byte = field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
    const float sc = mx4_scale(byte);
    uint32_t w = 0;
    if (byte != 255u) {
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], sc, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], sc, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], sc, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], sc, 3);
    }
    codes[i] = w;
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
  }
}

// One lane for each eight values.
template <bool BF>
__global__ __launch_bounds__(256) void dequantize(const uint32_t* __restrict__ codes,
                                                  const uint8_t* __restrict__ scales, int rows, int K,
                                                  bool vec, void* __restrict__ y) {
  const int nb = mx4_blocks(K);
  const long long n = (long long)rows * nb * 4;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = i / (nb * 4);
    const int c = (int)(i - r * (nb * 4)) * 8;
    const uint4 v = __builtin_bit_cast(uint4, mx4_frag(codes[i], mx4_scale(scales[i >> 2])));
    const uint32_t p[4] = {v.x, v.y, v.z, v.w};
    if (BF) {
      uint16_t* o = static_cast<uint16_t*>(y) + r * K + c;
      if (vec && c + 8 <= K) {
        *reinterpret_cast<uint4*>(o) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < K) o[j] = (uint16_t)(p[j / 2] >> (16 * (j & 1)));
      }
    } else {
      float* o = static_cast<float*>(y) + r * K + c;
      if (vec && c + 8 <= K) {
        reinterpret_cast<float4*>(o)[0] = make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
        reinterpret_cast<float4*>(o)[1] = make_float4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
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
  const dim3 g(grid_of((long long)rows * mx4_blocks(K) * 4));
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  const bool vec = rows_vec(x, ld, xdtype == 1 ? 2 : 4);
  if (xdtype == 1)
    MOE_LAUNCH("mx4_quantize", s, quantize<true>, g, dim3(256), 0, s, x, ld, rows, K, vec, c, scales);
  else
    MOE_LAUNCH("mx4_quantize", s, quantize<false>, g, dim3(256), 0, s, x, ld, rows, K, vec, c, scales);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int K, int ydtype,
                                 void* y, hipStream_t s) {
  const dim3 g(grid_of((long long)rows * mx4_blocks(K) * 4));
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  const bool vec = rows_vec(y, K, ydtype == 1 ? 2 : 4);
  if (ydtype == 1)
    MOE_LAUNCH("mx4_dequantize", s, dequantize<true>, g, dim3(256), 0, s, c, scales, rows, K, vec, y);
  else
    MOE_LAUNCH("mx4_dequantize", s, dequantize<false>, g, dim3(256), 0, s, c, scales, rows, K, vec, y);
  return hipGetLastError();
}

}  // namespace moe
