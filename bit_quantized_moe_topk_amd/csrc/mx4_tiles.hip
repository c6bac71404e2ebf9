// Products of many rows with a microscaled matrix on 32x32x16 matrix-core
// tiles (bf16 weights converted in registers, bf16 or float32 rows).
//
// A workgroup takes up to 128 rows of one group and a strip of its matrix;
// each wave owns 64 matrix rows. A wave converts its own weights right before
// the products that use them (four conversions for eight values, against up to
// four products). Bound by the matrix cores, and for a few rows a group by the
// matrix's bytes.
#include "mx4_tile.h"

namespace moe {
namespace {

constexpr int kTN = 256;   // matrix rows per tile of the general kernel: four waves across, two down
constexpr int kTK = 64;    // columns per stage: two blocks
constexpr int kThreads = 512;

// One stage's products: R runs of 32 rows, 64 matrix rows, 64 columns. Lane
// half h holds block h of the stage (codes c, scale sc), so product step kk
// takes values 8 kk .. + 7 of both blocks.
template <int R, int P>
__device__ inline void stage_products(const uint4* xs, int run0, const uint4 (&c)[2], const float (&sc)[2],
                                      floatx16_t (&acc)[2][2]) {
  const int lane = threadIdx.x & 63, hq = 4 * (lane >> 5), r = lane & 31;
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    bf16x8_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      w[j] = mx4_frag(kk == 0 ? c[j].x : kk == 1 ? c[j].y : kk == 2 ? c[j].z : c[j].w, sc[j]);
#pragma unroll
    for (int p = P - 1; p >= 0; --p)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bf16x8_t x = __builtin_bit_cast(bf16x8_t, xs[p * kTM * 8 + chunk_at(32 * (run0 + i) + r, hq + kk)]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j], x, acc[i][j], 0, 0, 0);
      }
  }
}

// Any K, stride and alignment, and float32 rows (P = 3 bf16 parts a value;
// bf16: 1). Rows pass through registers, zeros in place of columns past K: the
// values of the stage after next are asked for before a stage's products and
// go to LDS, split into their parts, before the next one's. The weights of the
// next stage wait in registers.
template <int P>
__global__ __launch_bounds__(kThreads, 2) void tiles_forward(Mx4Args a, bool vec) {
  __shared__ uint4 xs[2][P * kTM * 8];
  __shared__ Tiles tiles;
  const int strips = (a.N + kTN - 1) / kTN;
  const int items = tiles_init(tiles, *reinterpret_cast<TilesScratch*>(xs), a) * strips;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r = lane & 31, wn = wave & 3, wm = wave >> 2;
  const int nb = mx4_blocks(a.K), S = (nb + 1) / 2;
  __shared__ int slot;
  Deal deal{items, (int)gridDim.x, a.counter, &slot, 0u};
  deal.ask();
  for (int item = deal.first(), next = 0; item < items; item = next) {
    next = deal.answer(item);
    deal.ask();
    const TileInfo t = tile_of(tiles, a, item, items, strips, kTN);
    const int R = (t.M + 31) / 32, run0 = wm ? (R + 1) / 2 : 0;
    // this wave's weights: matrix rows n0 + 64 wn + 32 j + r (past N: the last one, not stored)
    const int live = t.n0 + 64 * wn >= a.N ? 0 : wm ? R / 2 : (R + 1) / 2;
    const uint4* wc[2];
    const uint8_t* ws[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const size_t row = (size_t)t.e * a.N + min(t.n0 + 64 * wn + 32 * j + r, a.N - 1);
      wc[j] = reinterpret_cast<const uint4*>(a.wc) + row * nb;
      ws[j] = a.ws + row * nb;
    }
    // rows of a stage: thread: row tid / 4, chunks 2 (tid % 4) and + 1
    const int m = tid >> 2, q0 = 2 * (tid & 3);
    const int xr = m < t.M ? mx4_row(a, t.s0 + m) : -1;
    const char* row = xr < 0 ? nullptr : static_cast<const char*>(a.x) + (size_t)xr * a.ldx * (P == 1 ? 2 : 4);
    uint4 v1[2];
    float v3[2][8];
    auto ask = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int k = s * kTK + 8 * (q0 + z);
        if constexpr (P == 1) {
          v1[z] = make_uint4(0, 0, 0, 0);
          if (row && k < a.K) v1[z] = load8_bf16(reinterpret_cast<const uint16_t*>(row), k, a.K, vec);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v3[z][i] = 0.f;
          if (row && k < a.K) load8_f32(reinterpret_cast<const float*>(row), k, a.K, vec, v3[z]);
        }
      }
    };
    auto put = [&](int b) __attribute__((always_inline)) {
      if (m >= 32 * R) return;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        if constexpr (P == 1) {
          xs[b][chunk_at(m, q0 + z)] = v1[z];
        } else {
          uint4 p0, p1, p2;
          split3x8(v3[z], p0, p1, p2);
          xs[b][chunk_at(m, q0 + z)] = p0;
          xs[b][kTM * 8 + chunk_at(m, q0 + z)] = p1;
          xs[b][2 * kTM * 8 + chunk_at(m, q0 + z)] = p2;
        }
      }
    };
    auto load_w = [&](int s, uint4 (&c)[2], uint32_t (&sc)[2]) __attribute__((always_inline)) {
      const int b = 2 * s + h;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        c[j] = make_uint4(0, 0, 0, 0);
        sc[j] = 0;
        if (live && b < nb) {
          c[j] = wc[j][b];
          sc[j] = ws[j][b];
        }
      }
    };
    floatx16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = floatx16_t{};
    uint4 c[2], cn[2];
    uint32_t e[2], en[2];
    ask(0);
    load_w(0, c, e);
    put(0);
    if (S > 1) ask(1);
    __syncthreads();
    auto run = [&](auto RR) __attribute__((always_inline)) {
      constexpr int RN = decltype(RR)::value;
      for (int s = 0; s < S; ++s) {
        if (s + 1 < S) {
          load_w(s + 1, cn, en);
          put((s + 1) & 1);
          if (s + 2 < S) ask(s + 2);
        }
        const float sc[2] = {mx4_scale(e[0]), mx4_scale(e[1])};
        if constexpr (RN > 0) stage_products<RN, P>(xs[s & 1], run0, c, sc, acc);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          c[j] = cn[j];
          e[j] = en[j];
        }
        __syncthreads();
      }
    };
    if (live == 2) run(std::integral_constant<int, 2>{});
    else if (live == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 0>{});
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < live) store_run(a, acc[i], t.s0 + 32 * (run0 + i), t.M - 32 * (run0 + i), t.n0 + 64 * wn);
  }
}

// ---- rows and matrix streamed through LDS ---------------------------------------
//
// The same products where rows can be read 16 bytes at a time and K is a
// multiple of 128. Eight waves, one workgroup per CU. Rows, codes and scales
// come by direct global-to-LDS loads in steps of 128 columns, double buffered:
// as soon as a step is read its buffer takes the step after next, so a load has
// a whole step to land, and the loads run on across tiles: the matrix cores
// wait for memory at the first tile alone. (With the codes loaded
// straight into registers one 64-column stage ahead, 32 bytes from each of 32
// matrix rows at a time, those loads took a quarter of the kernel's time.)
// The workgroup is WN waves across 64 WN matrix rows by 8 / WN waves down its
// 128 rows; each converts the weights it multiplies.

constexpr int kStep = 128;  // columns per step: four blocks

template <int WN>
struct StreamBuf {
  uint4 x[2][kTM * 8];        // two 64-column stages (chunk_at)
  uint4 w[64 * WN * 4];       // matrix row n: its four blocks, block c at position c ^ ((n >> 2) & 3)
};

// WIDE: scales come 16 a load, for four steps (a multiple of 16 blocks, aligned),
// and the rows' loads are not left out for runs that are not there: a load costs
// by the 128-byte lines that it touches, and one that repeats a row touches few
// (a chunk of 8,192 tokens: 433 us without both). Else four scales a step.
template <int WN, bool WIDE>
__global__ __launch_bounds__(512, 2) void tiles_stream(Mx4Args a) {
  constexpr int kRuns = WN / 2;  // runs of 32 rows per wave
  constexpr int kWL = WN / 2;    // code loads per wave and step (16 matrix rows each)
  constexpr int kS = WIDE ? 4 : 1;  // dwords of scales per load and matrix row
  __shared__ StreamBuf<WN> buf[2];
  __shared__ __attribute__((aligned(16))) uint32_t scales[2][64 * WN * kS];
  __shared__ Tiles tiles;
  constexpr int strip = 64 * WN;
  const int strips = (a.N + strip - 1) / strip;
  const int items = tiles_init(tiles, *reinterpret_cast<TilesScratch*>(buf), a) * strips;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r = lane & 31, wn = wave % WN, wm = wave / WN;
  const int nb = mx4_blocks(a.K), P = a.K / kStep;
  __shared__ int slot;
  Deal deal{items, (int)gridDim.x, a.counter, &slot, 0u};
  int item = deal.first();
  if (item >= items) return;
  deal.ask();
  int next = deal.answer(item);

  // load cursor: this lane's rows (rows 16 wave + 8 u + l / 8, chunk l % 8 of the stage as placed;
  // those past the tile's repeat its last, and are not stored) and matrix rows (8 WN wave + 16 i +
  // l / 4, block l % 4 as placed), and the bases that advance by steps
  uint32_t xoff[2], woff[kWL], soff;
  int xrows = 0;  // rows to load, in whole runs
  int lp = 0;     // step of its tile
  int ls = 1;     // place of the last scales asked for (WIDE; else a step's go with its buffer)
  const char *xbase, *wbase, *sbase;
  int row_next[2];
  auto row_of = [&](int u) { return 16 * wave + 8 * u + (lane >> 3); };
  auto fetch_rows = [&](const TileInfo& t) {  // the row numbers of a tile, to be used later
#pragma unroll
    for (int u = 0; u < 2; ++u) row_next[u] = max(mx4_row(a, t.s0 + min(row_of(u), t.M - 1)), 0);
  };
  auto aim = [&](const TileInfo& t) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int q = (lane & 7) ^ ((row_of(u) >> 1) & 7);
      xoff[u] = (uint32_t)row_next[u] * (uint32_t)(2 * a.ldx) + 16 * q;
    }
    xbase = static_cast<const char*>(a.x);
    xrows = (t.M + 31) & ~31;
    lp = 0;
    wbase = reinterpret_cast<const char*>(a.wc) + (size_t)t.e * a.N * nb * 16;
    sbase = reinterpret_cast<const char*>(a.ws) + (size_t)t.e * a.N * nb;
#pragma unroll
    for (int i = 0; i < kWL; ++i) {
      const int n = 8 * WN * wave + 16 * i + (lane >> 2);
      woff[i] = (uint32_t)min(t.n0 + n, a.N - 1) * (nb * 16) + 16 * ((lane & 3) ^ ((n >> 2) & 3));
    }
    soff = (uint32_t)min(t.n0 + 8 * WN * wave + lane, a.N - 1) * nb;
  };
  auto load = [&](int b) __attribute__((always_inline)) {
    StreamBuf<WN>& B = buf[b];
    if (WIDE || 16 * wave < xrows) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        stream16(xbase, xoff[u], lds_offset(B.x[0]) + 1024 * (2 * wave + u));
        stream16(xbase + 128, xoff[u], lds_offset(B.x[1]) + 1024 * (2 * wave + u));
      }
    }
    xbase += 256;
#pragma unroll
    for (int i = 0; i < kWL; ++i) stream16(wbase, woff[i], lds_offset(B.w) + 1024 * (kWL * wave + i));
    if constexpr (WIDE) {  // (WN 8: a matrix row a lane)
      if (lp % 4 == 0) {
        ls ^= 1;
        stream16(sbase + 4 * lp, soff, lds_offset(scales[ls]) + 1024 * wave);
      }
    } else if (lane < 8 * WN) {
      stream4(sbase + 4 * lp, soff, lds_offset(scales[b]) + 32 * WN * wave);
    }
    wbase += 64;
    ++lp;
  };

  int b = 0, cs = 1;  // cs: place of the scales in use
  TileInfo t = tile_of(tiles, a, item, items, strips, strip), tn = t;
  fetch_rows(t);
  aim(t);
  load(0);
  load(1);
  step_done();
  for (;;) {
    const bool more = next < items;
    if (more) {
      deal.ask();
      tn = tile_of(tiles, a, next, items, strips, strip);
      fetch_rows(tn);
    }
    const int live = min(max((t.M + 31) / 32 - kRuns * wm, 0), kRuns);
    floatx16_t acc[kRuns][2];
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = floatx16_t{};
    // one loop for each number of live runs (a switch inside the loop makes the compiler move accumulators)
    auto run = [&](auto LL) __attribute__((always_inline)) {
      constexpr int L = decltype(LL)::value;
      // A step's eight product steps of 16 columns (q: stage q / 4, step q % 4 of it). The operands
      // of one are read while the last one's products run, and those of the next step's first
      // while this step's last do, past the barrier: the matrix cores have work across it.
      uint32_t sw[2];
      uint4 c[2];
      bf16x8_t x[2][L > 0 ? L : 1];
      auto read_w = [&](int st, uint4 (&v)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) v[j] = buf[b].w[4 * (64 * wn + 32 * j + r) + ((2 * st + h) ^ ((r >> 2) & 3))];
      };
      auto read_x = [&](int q) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < L; ++i)
          x[q & 1][i] =
              __builtin_bit_cast(bf16x8_t, buf[b].x[q >> 2][chunk_at(32 * (kRuns * wm + i) + r, 4 * h + (q & 3))]);
      };
      auto read_first = [&](int p) __attribute__((always_inline)) {
        if (WIDE && p % 4 == 0) cs ^= 1;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          sw[j] = scales[WIDE ? cs : b][kS * (64 * wn + 32 * j + r) + (WIDE ? p & 3 : 0)] >> (8 * h);
        read_w(0, c);
        read_x(0);
      };
      auto products = [&](int q, const uint4 (&v)[2], const uint32_t (&e)[2]) __attribute__((always_inline)) {
        bf16x8_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[j] = mx4_frag((q & 3) == 0 ? v[j].x : (q & 3) == 1 ? v[j].y : (q & 3) == 2 ? v[j].z : v[j].w,
                          mx4_scale((e[j] >> (16 * (q >> 2))) & 255u));
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j], x[q & 1][i], acc[i][j], 0, 0, 0);
      };
      // next: the load that follows (0: two steps on; 1, 2: the next tile's first and second)
      auto step = [&](auto next, int p) __attribute__((always_inline)) {
        uint4 c1[2];
        const uint32_t e[2] = {sw[0], sw[1]};
        if constexpr (L > 0) {
#pragma unroll
          for (int q = 0; q < 7; ++q) {
            if (q == 2) read_w(1, c1);
            read_x(q + 1);
            products(q, q < 4 ? c : c1, e);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        // everything is read: the buffer takes the step after next, which has a step to land
        step_done();
        if (decltype(next)::value == 0 || more) {
          if (decltype(next)::value == 1) aim(tn);
          load(b);
        }
        b ^= 1;
        if constexpr (L > 0) {
          __builtin_amdgcn_sched_barrier(0);
          if (decltype(next)::value != 2) read_first(p + 1);
          products(7, c1, e);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      if constexpr (L > 0) read_first(0);
      else if (WIDE) cs ^= (P / 4) & 1;
      for (int p = 0; p < P - 2; ++p) step(std::integral_constant<int, 0>{}, p);
      step(std::integral_constant<int, 1>{}, P - 2);
      step(std::integral_constant<int, 2>{}, P - 1);
    };
    if (live == kRuns) run(std::integral_constant<int, kRuns>{});
    else if (kRuns > 3 && live == 3) run(std::integral_constant<int, kRuns < 3 ? 0 : 3>{});
    else if (kRuns > 2 && live == 2) run(std::integral_constant<int, kRuns < 2 ? 0 : 2>{});
    else if (kRuns > 1 && live == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 0>{});
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
      if (i < live)
        store_run(a, acc[i], t.s0 + 32 * (kRuns * wm + i), t.M - 32 * (kRuns * wm + i), t.n0 + 64 * wn);
    if (!more) break;
    next = deal.answer(next);
    t = tn;
  }
}

}  // namespace

hipError_t launch_mx4_tiles(Mx4Args a, hipStream_t s) {
  const bool vec = rows_vec(a.x, a.ldx, a.xdtype == 1 ? 2 : 4);
  // streamed: scales on four bytes, 32-bit offsets within one matrix and within the rows
  const bool even = a.xdtype == 1 && vec && a.K % kStep == 0 && a.K >= 2 * kStep &&
                    (reinterpret_cast<uintptr_t>(a.ws) & 3) == 0 && (long long)a.N * a.K < (1LL << 32) &&
                    (a.perm ? a.T : a.A) * a.ldx * 2 < (1LL << 32);
  const bool wide = a.K % 512 == 0 && (reinterpret_cast<uintptr_t>(a.ws) & 15) == 0;
  const long long tiles = mx4_row_tiles(a);
  const int cap = device_cus();
  // The widest strip that still gives every CU a tile: rows are read once a strip. Of groups some
  // stay empty, so with long rows, where a CU without a tile costs more than a tile too many, half
  // as many more are asked for (us in strips of 128, 256, 512, bf16, 512 experts and a shared one, 10 a token, a few
  // popular: [1024, 2048], 8 tokens 15, 20, 30, 16 tokens 26, 21, 31; [2048, 512], 4 tokens 12, 9, 14; evenly loaded,
  // [1024, 2048], 64 tokens 154, 117, 104, 8,192 tokens 607, 453, 415).
  int strip = even ? 512 : kTN;
  const int want = a.offsets && a.K >= 1024 ? cap + cap / 2 : cap;
  if (even && (tiles * ((a.N + 511) / 512) < want || a.N <= 256)) strip = 256;
  if (even && (tiles * ((a.N + 255) / 256) < want || a.N <= 128)) strip = 128;
  const long long most = ((long long)(a.A + kTM - 1) / kTM + (a.offsets ? a.E_tot : 0)) * ((a.N + strip - 1) / strip);
  const dim3 g((unsigned)(most < cap ? most : cap));
  if (most <= cap || g.x % kXcds) a.counter = nullptr;
  else if (a.counter) launch_mx4_zero(a.counter, s);
  if (!even && a.xdtype == 1) MOE_LAUNCH("mx4_tiles", s, tiles_forward<1>, g, dim3(kThreads), 0, s, a, vec);
  else if (!even) MOE_LAUNCH("mx4_tiles", s, tiles_forward<3>, g, dim3(kThreads), 0, s, a, vec);
  else if (strip == 512 && wide) MOE_LAUNCH("mx4_stream_512_wide", s, (tiles_stream<8, true>), g, dim3(512), 0, s, a);
  else if (strip == 512) MOE_LAUNCH("mx4_stream_512", s, (tiles_stream<8, false>), g, dim3(512), 0, s, a);
  else if (strip == 256) MOE_LAUNCH("mx4_stream_256", s, (tiles_stream<4, false>), g, dim3(512), 0, s, a);
  else MOE_LAUNCH("mx4_stream_128", s, (tiles_stream<2, false>), g, dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
