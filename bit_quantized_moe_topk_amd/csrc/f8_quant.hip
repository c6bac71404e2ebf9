// Quantisation to 8-bit codes with a float32 scale a block, and back (the
// format and the rounding: f8.h). One pass over the data: 16 lanes hold a block of a row, so its largest magnitude takes four
// lane steps and no LDS; a matrix block is one workgroup's registers. Bound by memory and, from cache, by
// the rounding: 8,192 bf16 rows of 2,048 values 13.4 us (50 MB, 3.8 TB/s; 14.8 with fourteen instructions a value in place of nine).
#include "f8.h"

namespace moe {
namespace {

// Rows: 16 lanes a block, eight values a lane.
template <bool BF>
__global__ __launch_bounds__(256) void quantize_rows(const void* __restrict__ x, long long ld, int rows, int K,
                                                     uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int nb = f8_blocks(K);
  const long long n = (long long)rows * nb * 16;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = n <= 0xFFFFFFFFLL ? (long long)((uint32_t)i / (uint32_t)(nb * 16)) : i / (nb * 16);
    const int c = (int)(i - r * (nb * 16)) * 8;
    float f[8], sc;
    load8<BF>(static_cast<const char*>(x) + r * ld * (BF ? 2 : 4), c, K, f);
    const uint2 q = f8_codes(f, f8_top16(f), &sc);
    *reinterpret_cast<uint2*>(codes + r * nb * kF8Block + c) = q;
    if ((threadIdx.x & 15) == 0) scales[i >> 4] = sc;
  }
}

// Matrices: a workgroup a block of 128 x 128; thread (row tid / 16 + 16 j, columns 8 (tid % 16) ..).
template <bool BF>
__global__ __launch_bounds__(256) void quantize_matrix(const void* __restrict__ x, long long ld, int rows, int K,
                                                       uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t most[4];
  const int nb = f8_blocks(K), rb = f8_blocks(rows), tid = threadIdx.x;
  const int kb = blockIdx.x % nb, b = blockIdx.x / nb, mat = b / rb, r0 = (b - mat * rb) * kF8Block;
  const int c = kb * kF8Block + 8 * (tid & 15);
  float f[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = r0 + 16 * j + (tid >> 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[j][i] = 0.f;
    if (r < rows) load8<BF>(static_cast<const char*>(x) + ((long long)mat * rows + r) * ld * (BF ? 2 : 4), c, K, f[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude(f[j][i]));
  }
  top = wave_reduce<true>(top);
  if ((tid & 63) == 0) most[tid >> 6] = top;
  __syncthreads();
  top = max(max(most[0], most[1]), max(most[2], most[3]));
  float sc = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = r0 + 16 * j + (tid >> 4);
    const uint2 q = f8_codes(f[j], top, &sc);
    if (r < rows) *reinterpret_cast<uint2*>(codes + ((long long)mat * rows + r) * nb * kF8Block + c) = q;
  }
  if (tid == 0) scales[((long long)mat * rb + r0 / kF8Block) * nb + kb] = sc;
}

template <bool BF>
__global__ __launch_bounds__(256) void dequantize(const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                                                  int mats, int rows, int K, int block_rows, void* __restrict__ y) {
  const int nb = f8_blocks(K), rb = (rows + block_rows - 1) / block_rows;
  const long long n = (long long)mats * rows * nb * 16;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long row = i / (nb * 16);
    const int c = (int)(i - row * (nb * 16)) * 8;
    if (c >= K) continue;
    const long long mat = row / rows, of = mat * rb + (row - mat * rows) / block_rows;
    const float s = scales[of * nb + c / kF8Block];
    const uint2 q = *reinterpret_cast<const uint2*>(codes + row * nb * kF8Block + c);
    float f[8];
    typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(z ? q.y : q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(z ? q.y : q.x, true);
      f[4 * z] = a.x * s;
      f[4 * z + 1] = a.y * s;
      f[4 * z + 2] = b.x * s;
      f[4 * z + 3] = b.y * s;
    }
    store8<BF>(static_cast<char*>(y) + row * K * (BF ? 2 : 4), c, K, f);
  }
}

unsigned blocks_for(long long n) {
  const long long g = (n + 255) / 256, most = 32LL * device_cus();
  return (unsigned)(g < most ? g : most);
}

}  // namespace

hipError_t launch_f8_quantize(const void* x, int xdtype, long long ld, int mats, int rows, int K, int block_rows,
                              uint8_t* codes, float* scales, hipStream_t s) {
  const int nb = f8_blocks(K);
  if (block_rows == 1) {
    const dim3 g(blocks_for((long long)mats * rows * nb * 16));
    if (xdtype == 1) MOE_LAUNCH("f8_quantize", s, quantize_rows<true>, g, dim3(256), 0, s, x, ld, mats * rows, K, codes, scales);
    else MOE_LAUNCH("f8_quantize", s, quantize_rows<false>, g, dim3(256), 0, s, x, ld, mats * rows, K, codes, scales);
  } else {
    const dim3 g((unsigned)((long long)mats * f8_blocks(rows) * nb));
    if (xdtype == 1) MOE_LAUNCH("f8_quantize_matrix", s, quantize_matrix<true>, g, dim3(256), 0, s, x, ld, rows, K, codes, scales);
    else MOE_LAUNCH("f8_quantize_matrix", s, quantize_matrix<false>, g, dim3(256), 0, s, x, ld, rows, K, codes, scales);
  }
  return hipGetLastError();
}

hipError_t launch_f8_dequantize(const uint8_t* codes, const float* scales, int mats, int rows, int K, int block_rows,
                                int ydtype, void* y, hipStream_t s) {
  const dim3 g(blocks_for((long long)mats * rows * f8_blocks(K) * 16));
  if (ydtype == 1) MOE_LAUNCH("f8_dequantize", s, dequantize<true>, g, dim3(256), 0, s, codes, scales, mats, rows, K, block_rows, y);
  else MOE_LAUNCH("f8_dequantize", s, dequantize<false>, g, dim3(256), 0, s, codes, scales, mats, rows, K, block_rows, y);
  return hipGetLastError();
}

}  // namespace moe
