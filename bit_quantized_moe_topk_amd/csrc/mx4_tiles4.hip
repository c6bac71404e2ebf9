// Products of many microscaled rows with a microscaled matrix: both operands go
// from memory through LDS to the 4-bit matrix cores as they are, 32x32x64 a
// product, with each block's scale applied by the product itself.
//
// Eight waves, one workgroup per CU, 128 rows by 256 matrix rows; a wave owns
// two runs of 32 rows and 64 matrix rows, so four operand reads from LDS feed
// four products. A step is 256 columns (eight blocks); three buffers, so that a
// load has two steps to land. The products of a step take half a microsecond:
// what bounds a full chip is bringing the operands to LDS.
#include "mx4_tile.h"

namespace moe {
namespace {

constexpr int kN4 = 256;      // matrix rows per tile
constexpr int kBlocks = 8;    // blocks per step
constexpr int kBufs = 3;
constexpr int kThreads4 = 512;

struct Buf4 {
  uint4 x[kTM * kBlocks];   // row m: its eight blocks, as chunk_at places them
  uint4 w[kN4 * kBlocks];
};

// Eight scale bytes from block b of a row of nb.
__device__ inline uint2 load_scales(const uint8_t* row, int b, int nb) {
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = b + i < nb ? row[b + i] : 0u;
  return make_uint2(v[0] | v[1] << 8 | v[2] << 16 | v[3] << 24, v[4] | v[5] << 8 | v[6] << 16 | v[7] << 24);
}

// How scales come. A direct load costs by the 128-byte lines that it touches,
// so the fewer loads bring a row's scales the better.
//   kBytes : a byte at a time through registers (any K), which also waits for
//            more than it needs
//   kQuads : four at a time (a multiple of four blocks, aligned), two loads a step
//   kWide  : sixteen at a time (a multiple of 16 blocks, aligned), a load for two
//            steps; what LDS is left holds up to kWideGroups groups' tiles
enum Scales { kBytes, kQuads, kWide };
constexpr int kWideGroups = 2040;

template <int S>
__global__ __launch_bounds__(kThreads4, 2) void tiles_mx4(Mx4Args a) {
  constexpr int kCodes = 4;                                         // direct loads a wave and step, of codes,
  constexpr int kScaleLoads = S == kQuads ? 2 : S == kWide ? 1 : 0;  // and of scales (kWide: every other step)
  constexpr int kRowsS = kTM + kN4;  // the rows' scales, then the matrix rows'
  __shared__ Buf4 buf[kBufs];
  // kWide: two places of 16 a row; else per buffer four blocks and four
  __shared__ __attribute__((aligned(16))) uint32_t scale[S == kWide ? 2 * 4 * kRowsS : kBufs * 2 * kRowsS];
  __shared__ TilesOf<S == kWide ? kWideGroups : MOE_MAX_E_DEV + 4> tiles;
  const int strips = (a.N + kN4 - 1) / kN4;
  const int items = tiles_init(tiles, *reinterpret_cast<TilesScratch*>(buf), a) * strips;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r = lane & 31, wn = wave & 3, wm = wave >> 2;
  const int nb = mx4_blocks(a.K), P = (nb + kBlocks - 1) / kBlocks;
  __shared__ int slot;
  Deal deal{items, (int)gridDim.x, a.counter, &slot, 0u};
  deal.ask();
  for (int item = deal.first(), next = 0; item < items; item = next) {
    next = deal.answer(item);
    deal.ask();
    const TileInfo t = tile_of(tiles, a, item, items, strips, kN4);
    // loads of a step: rows 16 wave + 8 u + l / 8 and matrix rows 32 wave + 8 u + l / 8, the block
    // that belongs at position l % 8; scales: row tid, or matrix row tid - 128
    uint32_t xoff[2], woff[4];
    const int q = lane & 7;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int m = 16 * wave + 8 * u + (lane >> 3);
      xoff[u] = (uint32_t)max(mx4_row(a, t.s0 + min(m, t.M - 1)), 0) * (uint32_t)(16 * nb);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) woff[u] = (uint32_t)min(t.n0 + 32 * wave + 8 * u + (lane >> 3), a.N - 1) * (16 * nb);
    const char* wbase = reinterpret_cast<const char*>(a.wc) + (size_t)t.e * a.N * nb * 16;
    const int sr = S != kBytes ? 48 * wave + min(lane, 47) : min(tid, kRowsS - 1);
    const uint8_t* srow = sr < kTM ? a.xs + (size_t)max(mx4_row(a, t.s0 + min(sr, t.M - 1)), 0) * nb
                                   : a.ws + ((size_t)t.e * a.N + min(t.n0 + sr - kTM, a.N - 1)) * nb;
    const bool rows = 16 * wave < ((t.M + 31) & ~31);  // whether this wave loads rows
    auto load = [&](int p) __attribute__((always_inline)) {
      Buf4& B = buf[p % kBufs];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!rows) break;
        const int m = 16 * wave + 8 * u + (lane >> 3);
        stream16(a.x, xoff[u] + 16 * min(kBlocks * p + (q ^ ((m >> 1) & 7)), nb - 1), lds_offset(B.x) + 1024 * (2 * wave + u));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int n = 32 * wave + 8 * u + (lane >> 3);
        stream16(wbase, woff[u] + 16 * min(kBlocks * p + (q ^ ((n >> 1) & 7)), nb - 1), lds_offset(B.w) + 1024 * (4 * wave + u));
      }
      uint32_t* sc = scale + (S == kWide ? (p >> 1 & 1) * 4 * kRowsS : p % kBufs * 2 * kRowsS);
      if constexpr (S == kWide) {
        if (p % 2 == 0 && lane < 48) stream16(srow + 8 * p, lds_offset(sc) + 768 * wave);
      } else if constexpr (S == kQuads) {
        if (lane < 48) {
#pragma unroll
          for (int z = 0; z < 2; ++z)
            stream4(srow + min(kBlocks * p + 4 * z, nb - 4), lds_offset(sc + z * kRowsS) + 192 * wave);
        }
      } else if (tid < kRowsS) {
        const uint2 v = load_scales(srow, kBlocks * p, nb);
        sc[tid] = v.x;
        sc[kRowsS + tid] = v.y;
      }
    };
    const int R = (t.M + 31) / 32, run0 = wm ? (R + 1) / 2 : 0, live = wm ? R / 2 : (R + 1) / 2;
    floatx16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = floatx16_t{};
    load(0);
    if (P > 1) load(1);
    // all but the last load(), of step p, have landed
    auto done = [&](int p) __attribute__((always_inline)) {
      if (p >= P) step_done();
      else if (S == kWide && p % 2) {
        if (rows) step_done<kCodes + 2>();
        else step_done<kCodes>();
      } else {
        if (rows) step_done<kCodes + 2 + kScaleLoads>();
        else step_done<kCodes + kScaleLoads>();
      }
    };
    done(1);
    for (int p = 0; p < P; ++p) {
      if (p + 2 < P) load(p + 2);  // into step p - 1's buffer, which every wave has left
      const Buf4& B = buf[p % kBufs];
      if (live > 0) {
        // blocks past the row's end repeat others: scales of 2^-127 for both operands make them add nothing
        const int left = nb - kBlocks * p;
        const uint32_t m0 = left >= 4 ? ~0u : (1u << 8 * left) - 1u;
        const uint32_t m1 = left >= 8 ? ~0u : left <= 4 ? 0u : (1u << 8 * (left - 4)) - 1u;
        uint2 sw[2], sx[2];
        const uint32_t* sc = scale + (S == kWide ? (p >> 1 & 1) * 4 * kRowsS : p % kBufs * 2 * kRowsS);
        auto scales_of = [&](int row) {
          const uint2 v = S == kWide ? *reinterpret_cast<const uint2*>(sc + 4 * row + 2 * (p & 1))
                                     : make_uint2(sc[row], sc[kRowsS + row]);
          return make_uint2(v.x & m0, v.y & m1);
        };
#pragma unroll
        for (int j = 0; j < 2; ++j) sw[j] = scales_of(kTM + 64 * wn + 32 * j + r);
#pragma unroll
        for (int i = 0; i < 2; ++i) sx[i] = scales_of(32 * min(run0 + i, 3) + r);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          int8v_t w[2], x[2];
          int ew[2], ex[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 v = B.w[chunk_at(64 * wn + 32 * j + r, 2 * s + h)];
            w[j] = int8v_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
            ew[j] = (int)((s < 2 ? sw[j].x : sw[j].y) >> (8 * h + 16 * (s & 1)));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i == 1 && live < 2) continue;
            const uint4 v = B.x[chunk_at(32 * (run0 + i) + r, 2 * s + h)];
            x[i] = int8v_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
            ex[i] = (int)((s < 2 ? sx[i].x : sx[i].y) >> (8 * h + 16 * (s & 1)));
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[j], x[i], acc[i][j], 4, 4, 0, ew[j], 0, ex[i]);
          }
        }
      }
      // the next step's loads have landed; this iteration's may be in flight
      done(p + 2);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < live) store_run(a, acc[i], t.s0 + 32 * (run0 + i), t.M - 32 * (run0 + i), t.n0 + 64 * wn);
  }
}

}  // namespace

// Offsets within the rows and within one matrix are 32 bits wide.
bool mx4_tiles4_can(const Mx4Args& a) {
  const long long row = 16LL * mx4_blocks(a.K);
  return a.xdtype == kMx4 && (a.perm ? a.T : a.A) * row < (1LL << 32) && a.N * row < (1LL << 32);
}

hipError_t launch_mx4_tiles4(Mx4Args a, hipStream_t s) {
  const int nb = mx4_blocks(a.K);
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.ws) | reinterpret_cast<uintptr_t>(a.xs);
  const long long strips = (a.N + kN4 - 1) / kN4;
  const long long most = ((long long)(a.A + kTM - 1) / kTM + (a.offsets ? a.E_tot : 0)) * strips;
  const int cap = device_cus();
  const dim3 g((unsigned)(most < cap ? most : cap));
  if (most <= cap || g.x % kXcds) a.counter = nullptr;
  else if (a.counter) launch_mx4_zero(a.counter, s);
  if (nb % 16 == 0 && at % 16 == 0 && a.E_tot <= kWideGroups)
    MOE_LAUNCH("mx4_tiles4_wide", s, tiles_mx4<kWide>, g, dim3(kThreads4), 0, s, a);
  else if (nb % 4 == 0 && at % 4 == 0)
    MOE_LAUNCH("mx4_tiles4_quads", s, tiles_mx4<kQuads>, g, dim3(kThreads4), 0, s, a);
  else
    MOE_LAUNCH("mx4_tiles4_bytes", s, tiles_mx4<kBytes>, g, dim3(kThreads4), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
