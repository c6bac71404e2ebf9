// Products of many 8-bit rows with an 8-bit matrix, and with the matrix turned
// (the gradient for the rows), on 16x16 matrix-core tiles with 128 columns a step.
//
// A step of the contraction is one block, so a product's 128 terms share two
// scales: the matrix cores add them up from zero, and one multiply-add a result
// brings the sum into the accumulator. A workgroup takes up to 128 rows of one
// group and a strip of 64 WN results a row; eight waves, WN across and 8 / WN
// down, own 64 results of 16 WN rows each. Rows, codes and scales come by direct
// global-to-LDS loads, three buffers, so that a load has two steps to land, and
// the loads run on across tiles.
//
// The turned matrix lies in LDS as it is stored, contraction rows of 256 (128)
// bytes, and is read with transposing loads: 16 lanes read 8 rows of 16 codes and
// get 8 codes of one column each.
#include "f8.h"

namespace moe {
namespace {

constexpr int kBufs = 3;
constexpr int kThreads = 512;
constexpr int kRun = 16;  // rows of a product

template <int WN>
struct Buf8 {
  uint4 x[kTM * 8];        // row m: its eight chunks of 16 codes, as chunk_at places them
  uint4 w[64 * WN * 8];    // matrix row n likewise; turned: contraction row c, its 4 WN chunks of 16 columns (turned_at)
};

// Place of chunk q of contraction row c: the eight rows that 16 lanes read take different banks, and so do
// the rows 32 further on that the next 16 lanes read.
template <int WN>
__device__ inline int turned_at(int c, int q) {
  return c * (4 * WN) + (q ^ (WN >= 4 ? (c & 7) | ((c >> 2) & 8) : (c & 7)));
}

__device__ inline void f8_store_bf16(const F8Args& a, const floatx4_t (&acc)[4], int row, bool there, int n0, bool wide) {
  const int g = (threadIdx.x & 63) >> 4;
  uint16_t* y = static_cast<uint16_t*>(a.y) + (size_t)row * a.N;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    uint32_t p[4];
    // each lane has four neighbours of tiles j and j + 1; rows of 16 lanes swap, so that each has eight of one tile
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const auto s = __builtin_amdgcn_permlane16_swap(pack_bf16(acc[j][2 * z], acc[j][2 * z + 1]),
                                                      pack_bf16(acc[j + 1][2 * z], acc[j + 1][2 * z + 1]), false, false);
      p[z] = s[0];
      p[2 + z] = s[1];
    }
    const int n = n0 + 16 * (j + (g & 1)) + 8 * (g >> 1);
    if (!there) continue;
    if (wide) {
      if (n < a.N) *reinterpret_cast<uint4*>(y + n) = make_uint4(p[0], p[1], p[2], p[3]);
    } else {
#pragma unroll
      for (int z = 0; z < 8; ++z)
        if (n + z < a.N) y[n + z] = (uint16_t)(p[z / 2] >> (16 * (z & 1)));
    }
  }
}

__device__ inline void f8_store_f32(const F8Args& a, const floatx4_t (&acc)[4], int row, bool there, int n0, bool wide) {
  const int g = (threadIdx.x & 63) >> 4;
  if (!there) return;
  float* y = static_cast<float*>(a.y) + (size_t)row * a.N;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = n0 + 16 * j + 4 * g;
    if (wide) {
      if (n < a.N) *reinterpret_cast<floatx4_t*>(y + n) = acc[j];
    } else {
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (n + z < a.N) y[n + z] = acc[j][z];
    }
  }
}

template <bool EXACT>
struct Frag {  // 32 codes of a lane, as its products take them
  int8v_t v;
  __device__ void set(const int8v_t& c) { v = c; }
  __device__ static floatx4_t product(const Frag& a, const Frag& b) { return f8_products<false>(a.v, b.v); }
};
template <>
struct Frag<true> {
  bf16x8_t v[4];
  __device__ void set(const int8v_t& c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f8_bf16(c[2 * i], c[2 * i + 1]);
  }
  __device__ static floatx4_t product(const Frag& a, const Frag& b) {
    floatx4_t c = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
  }
};

template <bool BACK, bool EXACT, int WN>
__global__ __launch_bounds__(kThreads, 2) void f8_tiles(F8Args a) {
  constexpr int kRuns = WN;             // runs of 16 rows a wave
  constexpr int kWL = WN;               // loads of the matrix a wave and step, 1 KB each
  constexpr int kLoads = 2 + kWL + 1;   // and of rows and their scales
  constexpr int strip = 64 * WN;
  __shared__ Buf8<WN> buf[kBufs];
  __shared__ float scale[kBufs][kTM];
  __shared__ Tiles tiles;
  __shared__ int slot;
  const int strips = (a.N + strip - 1) / strip;
  const int items = tiles_init(tiles, *reinterpret_cast<TilesScratch*>(buf), a) * strips;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4, wn = wave % WN, wm = wave / WN;
  const int P = max(a.xb, 2);  // (a contraction of one block has an empty second step)
  const int stored = BACK ? a.K : a.N;
  Deal deal{items, (int)gridDim.x, a.counter, &slot, 0u};
  int item = deal.first();
  if (item >= items) return;
  deal.ask();
  int next = deal.answer(item);

  // load cursor: rows 16 wave + 8 u + l / 8 of the tile, the chunk that belongs at position l % 8; row 16 wave + l of the scales
  const uint8_t *xp[2], *wp[kWL];
  const float* sp;
  int lp = 0, row_next[3];
  auto row_of = [&](int u) { return u < 2 ? 16 * wave + 8 * u + (lane >> 3) : 16 * wave + r; };
  auto fetch_rows = [&](const TileInfo& t) {  // the row numbers of a tile, to be used later
#pragma unroll
    for (int u = 0; u < 3; ++u) row_next[u] = max(mx4_row(a, t.s0 + min(row_of(u), t.M - 1)), 0);
  };
  auto aim = [&](const TileInfo& t) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      xp[u] = static_cast<const uint8_t*>(a.x) + (size_t)row_next[u] * a.xb * kF8Block + 16 * ((lane & 7) ^ ((row_of(u) >> 1) & 7));
    sp = a.xf + (size_t)row_next[2] * a.xb;
    const uint8_t* w = a.wc + (size_t)t.e * stored * a.wb * kF8Block;
#pragma unroll
    for (int u = 0; u < kWL; ++u) {
      if constexpr (BACK) {  // (the row is added a step at a time: past the last, the last again, against codes of 0)
        const int c = (16 * wave + 16 / kWL * u) + lane / (4 * WN), q = (lane % (4 * WN)) ^ (turned_at<WN>(c, 0) - c * 4 * WN);
        wp[u] = w + 16 * (size_t)min(t.n0 / 16 + q, 8 * a.wb - 1);
      } else {
        const int n = 8 * (WN * wave + u) + (lane >> 3);
        wp[u] = w + (size_t)min(t.n0 + n, a.N - 1) * a.wb * kF8Block + 16 * ((lane & 7) ^ ((n >> 1) & 7));
      }
    }
    lp = 0;
  };
  auto load = [&](int b) __attribute__((always_inline)) {
    Buf8<WN>& B = buf[b];
    const int p = min(lp, a.xb - 1);
#pragma unroll
    for (int u = 0; u < 2; ++u) stream16(xp[u] + (size_t)p * kF8Block, lds_offset(B.x) + 1024 * (2 * wave + u));
#pragma unroll
    for (int u = 0; u < kWL; ++u) {
      size_t at = (size_t)p * kF8Block;
      if constexpr (BACK)
        at = (size_t)min(p * kF8Block + 16 * wave + 16 / kWL * u + lane / (4 * WN), a.K - 1) * a.wb * kF8Block;
      stream16(wp[u] + at, lds_offset(B.w) + 1024 * (kWL * wave + u));
    }
    if (lane < 16) stream4(sp + p, lds_offset(scale[b]) + 64 * wave);
    ++lp;
  };

  int b = 0;
  TileInfo t = tile_of<kTM, kRun>(tiles, a, item, items, strips, strip), tn = t;
  fetch_rows(t);
  aim(t);
  load(0);
  load(1);
  step_done<kLoads>();
  for (;;) {
    const bool more = next < items;
    if (more) {
      deal.ask();
      tn = tile_of<kTM, kRun>(tiles, a, next, items, strips, strip);
      fetch_rows(tn);
    }
    // this wave's runs of rows: all runs, dealt over the waves down
    const int R = (t.M + kRun - 1) / kRun, of = 8 / WN;
    const int run0 = wm * R / of, live = t.n0 + 64 * wn < a.N ? (wm + 1) * R / of - run0 : 0;
    const float* ws = a.wf + (size_t)t.e * f8_blocks(stored) * a.wb +
                      (BACK ? (size_t)min((t.n0 + 64 * wn) / kF8Block, a.wb - 1) : (size_t)min((t.n0 + 64 * wn) / kF8Block, f8_blocks(a.N) - 1) * a.wb);
    const size_t wstep = BACK ? a.wb : 1;
    floatx4_t acc[kRuns][4];
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = floatx4_t{};
    auto run = [&](auto LL) __attribute__((always_inline)) {
      constexpr int L = decltype(LL)::value;
      for (int p = 0; p < P; ++p) {
        const int b2 = b == 0 ? 2 : b - 1;  // the buffer of the step before, which every wave has left
        const bool loads = p + 2 < P || more;
        if (p + 2 == P && more) aim(tn);
        if (loads) load(b2);
        if (L > 0 && p < a.xb) {
          const Buf8<WN>& B = buf[b];
          const float sw = ws[(size_t)p * wstep];
          Frag<EXACT> w[4];
          float s[L > 0 ? L : 1];
#pragma unroll
          for (int i = 0; i < L; ++i) s[i] = scale[b][kRun * (run0 + i) + r];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (BACK) {
              typedef int v2i __attribute__((ext_vector_type(2)));
              int8v_t v;
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const int c = 32 * g + 8 * z + (r >> 1);
                const char* from = reinterpret_cast<const char*>(B.w + turned_at<WN>(c, 4 * wn + j)) + 8 * (r & 1);
                const v2i u = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (__attribute__((address_space(3))) v2i*)(__attribute__((address_space(3))) char*)const_cast<char*>(from));
                v[2 * z] = u[0];
                v[2 * z + 1] = u[1];
              }
              w[j].set(v);
            } else {
              const int n = 64 * wn + 16 * j + r;
              w[j].set(f8_pair(B.w[chunk_at(n, 2 * g)], B.w[chunk_at(n, 2 * g + 1)]));
            }
          }
#pragma unroll
          for (int i = 0; i < L; ++i) {
            Frag<EXACT> x;
            const int m = kRun * (run0 + i) + r;
            x.set(f8_pair(B.x[chunk_at(m, 2 * g)], B.x[chunk_at(m, 2 * g + 1)]));
            const float f = s[i] * sw;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const floatx4_t c = Frag<EXACT>::product(w[j], x);
#pragma unroll
              for (int z = 0; z < 4; ++z) acc[i][j][z] = fmaf(c[z], f, acc[i][j][z]);
            }
          }
        }
        // the next step's loads have landed; this iteration's may be in flight
        if (loads) step_done<kLoads>();
        else step_done();
        b = b == 2 ? 0 : b + 1;
      }
    };
    if (live == 4) run(std::integral_constant<int, kRuns < 4 ? 0 : 4>{});
    else if (live == 3) run(std::integral_constant<int, kRuns < 3 ? 0 : 3>{});
    else if (live == 2) run(std::integral_constant<int, kRuns < 2 ? 0 : 2>{});
    else if (live == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 0>{});
    const bool wide = a.N % (a.ydtype == 1 ? 8 : 4) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
      if (i < live) {
        const int m = kRun * (run0 + i) + r;
        if (a.ydtype == 1) f8_store_bf16(a, acc[i], t.s0 + m, m < t.M, t.n0 + 64 * wn, wide);
        else f8_store_f32(a, acc[i], t.s0 + m, m < t.M, t.n0 + 64 * wn, wide);
      }
    if (!more) break;
    next = deal.answer(next);
    t = tn;
  }
}

}  // namespace

hipError_t launch_f8_tiles(F8Args a, hipStream_t s) {
  constexpr int strip = 256;
  const long long most = ((long long)(a.A + kTM - 1) / kTM + (a.offsets ? a.E_tot : 0)) * ((a.N + strip - 1) / strip);
  const int cap = device_cus();
  const dim3 g((unsigned)(most < cap ? most : cap));
  if (most <= cap || g.x % kXcds) a.counter = nullptr;
  else if (a.counter) launch_mx4_zero(a.counter, s);
  if (a.back && a.exact) MOE_LAUNCH("f8_tiles_back", s, (f8_tiles<true, true, 4>), g, dim3(kThreads), 0, s, a);
  else if (a.back) MOE_LAUNCH("f8_tiles_back", s, (f8_tiles<true, false, 4>), g, dim3(kThreads), 0, s, a);
  else if (a.exact) MOE_LAUNCH("f8_tiles", s, (f8_tiles<false, true, 4>), g, dim3(kThreads), 0, s, a);
  else MOE_LAUNCH("f8_tiles", s, (f8_tiles<false, false, 4>), g, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
