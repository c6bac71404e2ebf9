// Products of groups of few rows, on 16x16x32 matrix-core tiles.
//
// With a handful of rows a group, a product is its matrices' bytes, each read
// once: so the matrix goes from memory straight to registers, a stage of
// columns ahead, by waves that wait for nothing else. Each owns 32 matrix rows
// over all of K, so no sums meet. A workgroup takes up to 16 rows of one group,
// staged in LDS (float32 rows as three exact bf16 parts, split once for all
// waves) while the last stage's products run, and goes on across tiles. 64
// tokens x 11 float32 rows, 512 experts, a few of them popular, [2048, 512]: 19
// us, what reading the matrices takes (37 us in 128-row tiles). Few tiles are
// bound by one wave's way through all columns, 1.5 us a stage of 256 for bf16
// rows.
#include "mx4_tile.h"

namespace moe {
namespace {

constexpr int kFew = 16;  // rows per tile

// One stage of a lane: codes and scales of C blocks for two matrix rows, and its share of the rows.
template <int P, int C, int X>
struct FewRegs {
  uint4 c[C][2];
  uint32_t s[C][2];
  uint4 x[X][P == 1 ? 1 : 2];
  int k;  // first column of the rows' share; past K: zeros
};

// P: bf16 parts of a value (1: bf16 rows, 3: float32 rows); C: chunks of 128 columns per stage; W: waves.
template <int P, int C, int W, bool VEC>
__global__ __launch_bounds__(64 * W, 4) void tiles_few(Mx4Args a) {
  constexpr int kThreads = 64 * W, kPieces = 16 * C;  // 16-byte pieces of a row and stage
  constexpr int kPer = kThreads / kFew, kX = kPieces / kPer;  // threads a row, pieces a thread
  __shared__ uint4 xs[2][P][kFew * kPieces];  // piece q of row m at q ^ m: 16 rows' reads of one piece hit all banks
  __shared__ Tiles tiles;
  __shared__ TilesScratch scratch;
  constexpr int strip = 32 * W;
  const int strips = (a.N + strip - 1) / strip;
  const int items = tiles_init<kFew>(tiles, scratch, a) * strips;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4, m = tid / kPer, q0 = tid % kPer;
  const int nb = mx4_blocks(a.K), S = (nb + 4 * C - 1) / (4 * C);
  auto tile = [&](int item) {
    TileInfo t;
    const int ti = item / strips;
    int end = a.A;
    t.e = 0;
    t.s0 = kFew * ti;
    if (a.offsets) {
      t.e = __builtin_amdgcn_readfirstlane(tile_group(tiles, a.E_tot, ti));
      t.s0 = __builtin_amdgcn_readfirstlane(scratch.first[t.e] + kFew * (ti - tiles.base[t.e]));
      end = __builtin_amdgcn_readfirstlane(scratch.first[t.e + 1]);
    }
    t.M = min(kFew, end - t.s0);
    t.n0 = (item - ti * strips) * strip;
    return t;
  };
  int ahead = blockIdx.x;
  if (ahead >= items) return;

  // load cursor: stage ls of tile t; the tile after it, and which of x's rows this thread brings of that
  int ls = S, id = 0;
  TileInfo t, ta;
  const uint4* wc[2];
  const uint8_t* ws[2];
  const char* xrow = nullptr;
  bool none = true;  // no such row
  auto look = [&]() {
    if (ahead >= items) return;
    ta = tile(ahead);
    if (a.perm) id = a.perm[ta.s0 + min(m, ta.M - 1)];  // (looked at when the tile's turn comes)
  };
  look();
  typedef FewRegs<P, C, kX> Regs;
  // Its loads are issued in any case (repeating some when there is no next stage): with a way past
  // them the compiler would make the products wait for them instead of for the last ones.
  auto load = [&](Regs& v) __attribute__((always_inline)) {
    const bool more = ls < S || ahead < items;
    if (ls == S && more) {
      t = ta;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const size_t row = (size_t)t.e * a.N + min(t.n0 + 32 * wave + 16 * j + r, a.N - 1);
        wc[j] = reinterpret_cast<const uint4*>(a.wc) + row * nb;
        ws[j] = a.ws + row * nb;
      }
      const int row = a.perm ? mx4_token(a, id) : t.s0 + min(m, t.M - 1);
      none = m >= t.M || row < 0;  // past the tile, or an id out of range
      xrow = static_cast<const char*>(a.x) + (size_t)(none ? 0 : row) * a.ldx * (P == 1 ? 2 : 4);
      ls = 0;
      ahead += gridDim.x;
      look();
    }
    v.k = none ? a.K : 128 * C * ls + 8 * q0;
#pragma unroll
    for (int z = 0; z < kX; ++z) {
      const int k = 128 * C * ls + 8 * (q0 + kPer * z);
      if constexpr (VEC) {
        const uint4* p = reinterpret_cast<const uint4*>(xrow + (size_t)min(k, a.K - 8) * (P == 1 ? 2 : 4));
        v.x[z][0] = p[0];
        if constexpr (P > 1) v.x[z][1] = p[1];
      } else if constexpr (P == 1) {
        if (k < a.K) v.x[z][0] = load8_bf16(reinterpret_cast<const uint16_t*>(xrow), k, a.K, false);
      } else {
        float f[8];
        if (k < a.K) load8_f32(reinterpret_cast<const float*>(xrow), k, a.K, false, f);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v.x[z][i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                 __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
      }
    }
#pragma unroll
    for (int z = 0; z < C; ++z) {
      const int b = min(4 * (C * ls + z) + g, nb - 1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v.c[z][j] = wc[j][b];
        v.s[z][j] = ws[j][b];
      }
    }
    ls += more;
    return more;
  };
  int b = 0, cs = 0;  // LDS buffer and stage whose turn it is
  auto put = [&](const Regs& v, int to) __attribute__((always_inline)) {
#pragma unroll
    for (int z = 0; z < kX; ++z) {
      const int at = m * kPieces + ((q0 + kPer * z) ^ m);
      const bool there = v.k + 8 * kPer * z < a.K;
      uint4 x[P == 1 ? 1 : 2];
#pragma unroll
      for (int i = 0; i < (P == 1 ? 1 : 2); ++i) x[i] = there ? v.x[z][i] : make_uint4(0, 0, 0, 0);
      if constexpr (P == 1) {
        xs[to][0][at] = x[0];
      } else {
        const float f[8] = {__uint_as_float(x[0].x), __uint_as_float(x[0].y), __uint_as_float(x[0].z),
                            __uint_as_float(x[0].w), __uint_as_float(x[P > 1].x), __uint_as_float(x[P > 1].y),
                            __uint_as_float(x[P > 1].z), __uint_as_float(x[P > 1].w)};
        split3x8(f, xs[to][0][at], xs[to][P > 1 ? 1 : 0][at], xs[to][P > 1 ? 2 : 0][at]);
      }
    }
  };
  auto meet = [] { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  floatx4_t acc[2] = {};
  auto step = [&](const Regs& v, Regs& next) __attribute__((always_inline)) {
    const TileInfo now = t;
    const bool more = load(next);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int z = 0; z < C; ++z) {
      if (4 * (C * cs + z) >= nb) break;
      const bool there = 4 * (C * cs + z) + g < nb;  // a block past the row's end repeats its last: scale 2^-127, rows 0
      const float sc[2] = {mx4_scale(there ? v.s[z][0] : 0u), mx4_scale(there ? v.s[z][1] : 0u)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bf16x8_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 c = v.c[z][j];
          w[j] = mx4_frag(i == 0 ? c.x : i == 1 ? c.y : i == 2 ? c.z : c.w, sc[j]);
        }
#pragma unroll
        for (int p = P - 1; p >= 0; --p) {
          const bf16x8_t x = __builtin_bit_cast(bf16x8_t, xs[b][p][r * kPieces + ((4 * (4 * z + g) + i) ^ r)]);
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], x, acc[j], 0, 0, 0);
        }
      }
    }
    if (++cs == S) {  // acc[j][i]: matrix row 16 j + 4 g + i, row r
      cs = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = now.n0 + 32 * wave + 16 * j + 4 * g;
        const size_t at = (size_t)(now.s0 + r) * a.N + n;
        const bool whole = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
        if (r < now.M && n < a.N) {
          if (a.ydtype == 1) {
            uint16_t* y = static_cast<uint16_t*>(a.y) + at;
            const uint32_t lo = pack_bf16(acc[j][0], acc[j][1]), hi = pack_bf16(acc[j][2], acc[j][3]);
            if (whole) {
              *reinterpret_cast<uint2*>(y) = make_uint2(lo, hi);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n + i < a.N) y[i] = (uint16_t)((i < 2 ? lo : hi) >> (16 * (i & 1)));
            }
          } else {
            float* y = static_cast<float*>(a.y) + at;
            if (whole) {
              *reinterpret_cast<floatx4_t*>(y) = acc[j];
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n + i < a.N) y[i] = acc[j][i];
            }
          }
        }
        acc[j] = floatx4_t{};
      }
    }
    if (more) put(next, b ^ 1);
    meet();
    b ^= 1;
    return more;
  };
  Regs even, odd;
  load(even);
  put(even, 0);
  meet();
  while (step(even, odd) && step(odd, even)) {
  }
}

}  // namespace

hipError_t launch_mx4_few(const Mx4Args& a, hipStream_t s) {
  const bool vec = a.K % 8 == 0 && rows_vec(a.x, a.ldx, a.xdtype == 1 ? 2 : 4);
  const int strip = a.xdtype == 1 ? 128 : 256;
  const long long groups = !a.offsets ? 0 : a.A < a.E_tot ? a.A : a.E_tot;
  const long long most = (((long long)a.A + kFew - 1) / kFew + groups) * ((a.N + strip - 1) / strip);
  const long long cap = (a.xdtype == 1 ? 4 : 2) * (long long)device_cus();
  const dim3 g((unsigned)(most < cap ? most : cap));
  if (a.xdtype == 1 && vec) MOE_LAUNCH("mx4_few", s, (tiles_few<1, 2, 4, true>), g, dim3(256), 0, s, a);
  else if (a.xdtype == 1) MOE_LAUNCH("mx4_few", s, (tiles_few<1, 2, 4, false>), g, dim3(256), 0, s, a);
  else if (vec) MOE_LAUNCH("mx4_few", s, (tiles_few<3, 2, 8, true>), g, dim3(512), 0, s, a);
  else MOE_LAUNCH("mx4_few", s, (tiles_few<3, 2, 8, false>), g, dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
