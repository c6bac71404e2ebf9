// Products of many 8-bit rows with an 8-bit matrix, and with the matrix turned
// (the gradient for the rows), on 16x16 matrix-core tiles with 128 columns a step.
//
// A step of the contraction is one block, so a product's 128 terms share two
// scales: the matrix cores add them up from zero, and one multiply-add a result
// brings the sum into the accumulator. A workgroup takes up to TM rows of one
// group and a strip of 64 WN results a row; eight waves, WN across and 8 / WN
// down, own 64 results of TM WN / 8 rows each. Rows, codes and scales come by direct
// global-to-LDS loads that run on across tiles, three buffers of the matrix and two
// or three of rows. A wave reads the next step's operands into the registers of
// those that its products have used up, so a buffer is free for the load of three
// (two) steps on when its step begins, and the matrix cores run through the
// barrier between steps.
//
// Bound, one matrix: by the matrix cores and the LDS reads that feed them: 8192 x
// 1024 x 8192 (rows, results, columns) 77 us, 1.78 PFLOP/s, where a large library
// product in 8 bits reaches 2.7; with 2,048 columns 25 us, as the first loads and
// the stores of 256 tiles, one a CU, are not covered. Grouped: by the loads into
// LDS: 8,192 tokens to 10 of 512 experts and a shared one, [1024, 2048], 313 to 328 us,
// 1.15 PFLOP/s (at 379 us: 346 without the products, 223 without the loads); the
// gradient of 1,024 tokens 227 us, at a copy's rate of 5.1 TB/s.
// Tried without gain: beginning each tile's contraction at another column (377 of
// 379), scales 16 bytes at a time, loading only the rows that are there, 2 to 8
// products between one and the addition of its sum (within 3 %).
//
// The turned matrix lies in LDS as it is stored, contraction rows of 256 (128)
// bytes, and is read with transposing loads: 16 lanes read 8 rows of 16 codes and
// get 8 codes of one column each.
#include "f8.h"

namespace moe {
namespace {

constexpr int kWBufs = 3;
// Buffers of rows: as many as LDS has room for. Products between one and the addition of its sum: as many as registers hold.
constexpr int xbufs(int TM) { return TM <= 128 ? 3 : 2; }
constexpr int lag(int TM) { return TM <= 128 ? 4 : 2; }
constexpr int kThreads = 512;
constexpr int kRun = 16;  // rows of a product

template <int WN, int TM>
struct Bufs8 {
  uint4 w[kWBufs][64 * WN * 8];  // matrix row n: its eight chunks of 16 codes, as chunk_at places them; turned: contraction
                                 // row c, its 4 WN chunks of 16 columns (turned_at)
  uint4 x[xbufs(TM)][TM * 8];       // row m, as chunk_at places it
};

// A lane's 32 codes of a row of 128 are chunks g and g + 4, g = l / 16. (A 16-byte read serves lanes 0-3, 12-15 and 20-27 at
// once, and so on: with chunks g and g + 1 beside one another those hit all banks once, with 2 g and 2 g + 2 twice, which
// took 8 cycles a read instead of 4.)
// Place of chunk q of contraction row c: the eight rows that 16 lanes read take different banks, and so do
// the rows 16 further on that the next 16 lanes read.
template <int WN>
__device__ inline int turned_at(int c, int q) {
  return c * (4 * WN) + (q ^ (WN >= 4 ? (c & 7) | (((c >> 4) ^ (c >> 5)) & 1) << 3 : (c & 7)));
}

__device__ inline void f8_store_bf16(const F8Args& a, const floatx4_t (&acc)[4], int row, bool there, int n0) {
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
    if (there) store8_bf16(y, n0 + 16 * (j + (g & 1)) + 8 * (g >> 1), a.N, p[0], p[1], p[2], p[3]);
  }
}

__device__ inline void f8_store_f32(const F8Args& a, const floatx4_t (&acc)[4], int row, bool there, int n0) {
  const int g = (threadIdx.x & 63) >> 4;
  float* y = static_cast<float*>(a.y) + (size_t)row * a.N;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (there) store4_f32(y, n0 + 16 * j + 4 * g, a.N, acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
}

// What a wave's products of a step read: 32 codes a lane of four runs of 16 matrix rows and of L runs of rows, and the
// rows' scales.
template <int L>
struct Operands {
  int8v_t w[4], x[L > 0 ? L : 1];
  float s[L > 0 ? L : 1];
};

// A uniform value that no kernel of this launch writes, by a scalar load.
__device__ inline float uniform_load(const float* p) {
  return *(const __attribute__((address_space(4))) float*)(uintptr_t)p;
}

template <bool BACK, bool EXACT, int WN, int TM>
__global__ __launch_bounds__(kThreads, 2) void f8_tiles(F8Args a) {
  constexpr int kRuns = TM / kRun * WN / 8;  // runs of rows a wave
  constexpr int kWL = WN;                    // loads of the matrix a wave and step, 1 KB each
  constexpr int kXR = TM / 8, kXL = kXR / 8;  // rows that a wave loads, and its loads of them
  constexpr int kXBufs = xbufs(TM), kLag = lag(TM);
  constexpr int strip = 64 * WN;
  __shared__ Bufs8<WN, TM> buf;
  __shared__ float scale[kXBufs][TM];
  __shared__ Tiles tiles;
  __shared__ int slot;
  const int strips = (a.N + strip - 1) / strip;
  const int items = tiles_init<TM>(tiles, *reinterpret_cast<TilesScratch*>(&buf), a) * strips;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4, wn = wave % WN, wm = wave / WN;
  const int P = max(a.xb, 3);  // (a short contraction has empty steps: loads run three ahead, into the next tile at most)
  const int stored = BACK ? a.K : a.N;
  Deal deal{items, (int)gridDim.x, a.counter, &slot, 0u};
  int item = deal.first();
  if (item >= items) return;
  deal.ask();
  int next = deal.answer(item);

  // Two load cursors, of rows and of the matrix, the latter a step ahead. Rows: 8 of kXR wave .. a load, lane l / 8's, the chunk
  // that belongs at position l % 8; a row's scale a lane. Matrix: rows 8 (WN wave + u) + l / 8, or the columns of a contraction
  // row. Offsets of a lane, bases of all.
  uint32_t xoff[kXL], woff[kWL], soff;
  const uint8_t* wbase;
  int xq = 0, wq = 0, row_next[kXL + 1];
  auto row_of = [&](int u) { return kXR * wave + (u < kXL ? 8 * u + (lane >> 3) : min(lane, kXR - 1)); };
  auto fetch_rows = [&](const TileInfo& t) {  // the row numbers of a tile, to be used later
#pragma unroll
    for (int u = 0; u <= kXL; ++u) row_next[u] = max(mx4_row(a, t.s0 + min(row_of(u), t.M - 1)), 0);
  };
  const uint32_t xrow = (uint32_t)a.xb * kF8Block, wrow = (uint32_t)a.wb * kF8Block;
  auto turned_row = [&](int u) { return 16 * wave + 16 / kWL * u + lane / (4 * WN); };
  auto aim_rows = [&]() {
#pragma unroll
    for (int u = 0; u < kXL; ++u) xoff[u] = (uint32_t)row_next[u] * xrow + 16 * ((lane & 7) ^ ((row_of(u) >> 1) & 7));
    soff = (uint32_t)row_next[kXL] * (uint32_t)a.xb * 4u;
    xq = 0;
  };
  auto aim_matrix = [&](const TileInfo& t) {
    wbase = a.wc + (size_t)t.e * stored * wrow;
#pragma unroll
    for (int u = 0; u < kWL; ++u) {
      if constexpr (BACK) {  // (the row is added a step at a time: past the last, the last again, against codes of 0)
        const int c = turned_row(u), q = (lane % (4 * WN)) ^ (turned_at<WN>(c, 0) - c * 4 * WN);
        woff[u] = 16u * (uint32_t)min(t.n0 / 16 + q, 8 * a.wb - 1);
      } else {
        const int n = 8 * (WN * wave + u) + (lane >> 3);
        woff[u] = (uint32_t)min(t.n0 + n, a.N - 1) * wrow + 16 * ((lane & 7) ^ ((n >> 1) & 7));
      }
    }
    wq = 0;
  };
  auto load_rows = [&](int at) __attribute__((always_inline)) {
    const int p = min(xq, a.xb - 1);
#pragma unroll
    for (int u = 0; u < kXL; ++u)
      stream16(static_cast<const uint8_t*>(a.x) + p * kF8Block, xoff[u], lds_offset(buf.x[at]) + 1024 * (kXL * wave + u));
    if (lane < kXR) stream4(a.xf + p, soff, lds_offset(scale[at]) + 4 * kXR * wave);
    ++xq;
  };
  auto load_matrix = [&](int at) __attribute__((always_inline)) {
    const int p = min(wq, a.xb - 1);
#pragma unroll
    for (int u = 0; u < kWL; ++u) {
      if constexpr (BACK)
        stream16(wbase, woff[u] + (uint32_t)min(p * kF8Block + turned_row(u), a.K - 1) * wrow, lds_offset(buf.w[at]) + 1024 * (kWL * wave + u));
      else
        stream16(wbase + p * kF8Block, woff[u], lds_offset(buf.w[at]) + 1024 * (kWL * wave + u));
    }
    ++wq;
  };
  // A step asks for rows kXBufs steps on, then for the matrix three steps on: all but the loads of three steps on have landed,
  // and every wave has come here.
  auto done = [](bool loads) __attribute__((always_inline)) {
    if (loads) step_done<kWL + (kXBufs == 3 ? kXL + 1 : 0)>();
    else step_done();
  };

  int b = 0, x = 0;  // the running step's buffers
  TileInfo t = tile_of<TM, kRun>(tiles, a, item, items, strips, strip), tn = t;
  fetch_rows(t);
  aim_rows();
  aim_matrix(t);
  load_rows(0);
  load_rows(1);
  if (kXBufs == 3) load_rows(2);
  load_matrix(0);
  load_matrix(1);
  load_matrix(2);
  step_done<kWL>();
  for (;;) {
    const bool more = next < items;
    if (more) {
      deal.ask();
      tn = tile_of<TM, kRun>(tiles, a, next, items, strips, strip);
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
    // one loop for each number of live runs (a switch inside the loop makes the compiler move accumulators)
    auto run = [&](auto LL) __attribute__((always_inline)) {
      constexpr int L = decltype(LL)::value;
      auto read_scales = [&](Operands<L>& o, int at) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < L; ++i) o.s[i] = scale[at][kRun * (run0 + i) + r];
      };
      auto read_w = [&](Operands<L>& o, int at, int j) __attribute__((always_inline)) {
        if constexpr (BACK) {
          typedef int v2i __attribute__((ext_vector_type(2)));
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int c = 16 * g + 8 * (z & 1) + 64 * (z >> 1) + (r >> 1);
            const char* from = reinterpret_cast<const char*>(buf.w[at] + turned_at<WN>(c, 4 * wn + j)) + 8 * (r & 1);
            const v2i u = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) v2i*)(__attribute__((address_space(3))) char*)const_cast<char*>(from));
            o.w[j][2 * z] = u[0];
            o.w[j][2 * z + 1] = u[1];
          }
        } else {
          const int n = 64 * wn + 16 * j + r;
          o.w[j] = f8_pair(buf.w[at][chunk_at(n, g)], buf.w[at][chunk_at(n, g + 4)]);
        }
      };
      auto read_x = [&](Operands<L>& o, int at, int i) __attribute__((always_inline)) {
        const int m = kRun * (run0 + i) + r;
        o.x[i] = f8_pair(buf.x[at][chunk_at(m, g)], buf.x[at][chunk_at(m, g + 4)]);
      };
      float sw = 0.f;
      const float* wp = ws;
      // Step p, while the next step's operands take the places of those that are used up and loads are on their way. A
      // block's sum is brought into its accumulator kLag products later, when it is there.
      Operands<L> o;
      auto step = [&](int p, bool loads) __attribute__((always_inline)) {
        const int b1 = b == kWBufs - 1 ? 0 : b + 1;
        float f[L > 0 ? L : 1];
#pragma unroll
        for (int i = 0; i < L; ++i) f[i] = p < a.xb ? o.s[i] * sw : 0.f;
        if (loads || p + kXBufs < P) load_rows(x);
        if (loads) load_matrix(b);
        x = x == kXBufs - 1 ? 0 : x + 1;
        if constexpr (L > 0) {
          if (p + 1 < a.xb) wp += wstep;
          sw = uniform_load(wp);
          read_scales(o, x);
          __builtin_amdgcn_sched_barrier(0);
          floatx4_t c[kLag + 1];
#pragma unroll
          for (int k = 0; k < 4 * L + kLag; ++k) {
            if (k < 4 * L) c[k % (kLag + 1)] = f8_products<false>(o.w[k % 4], o.x[k / 4]);
            if (k < 4 * L && k >= 4 * L - 4) read_w(o, b1, k % 4);
            if (k < 4 * L && k % 4 == 3) read_x(o, x, k / 4);
            if (k >= kLag) {
              const int i = (k - kLag) / 4, j = (k - kLag) % 4;
#pragma unroll
              for (int z = 0; z < 4; ++z) acc[i][j][z] = fmaf(c[(k - kLag) % (kLag + 1)][z], f[i], acc[i][j][z]);
              asm volatile("" : "+v"(acc[i][j]));  // here, not past the step's end, where the compiler moves it with all the sums
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        done(loads);
        b = b1;
      };
      // The same with bf16 products: codes become bf16 as they are read, which leaves no registers for a second set; the
      // step's buffer is loaded again when every wave has read it.
      auto step_exact = [&](int p) __attribute__((always_inline)) {
        if (L > 0 && p < a.xb) {
          read_scales(o, x);
          const float swp = uniform_load(wp);
          wp += wstep;
          bf16x8_t w[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            read_w(o, b, j);
#pragma unroll
            for (int z = 0; z < 4; ++z) w[j][z] = f8_bf16(o.w[j][2 * z], o.w[j][2 * z + 1]);
          }
#pragma unroll
          for (int i = 0; i < L; ++i) {
            read_x(o, x, i);
            bf16x8_t v[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] = f8_bf16(o.x[i][2 * z], o.x[i][2 * z + 1]);
            const float f = o.s[i] * swp;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              floatx4_t c = {};
#pragma unroll
              for (int z = 0; z < 4; ++z) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j][z], v[z], c, 0, 0, 0);
#pragma unroll
              for (int z = 0; z < 4; ++z) acc[i][j][z] = fmaf(c[z], f, acc[i][j][z]);
            }
          }
        }
        done(p + 2 < P || more);
        if (p + kXBufs == P && more) aim_rows();
        if (p + kXBufs < P || more) load_rows(x);
        if (p + 3 == P && more) aim_matrix(tn);
        if (p + 3 < P || more) load_matrix(b);
        b = b == kWBufs - 1 ? 0 : b + 1;
        x = x == kXBufs - 1 ? 0 : x + 1;
      };
      if constexpr (EXACT) {
        for (int p = 0; p < P; ++p) step_exact(p);
      } else {
        if constexpr (L > 0) {
          sw = uniform_load(wp);
          read_scales(o, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) read_w(o, b, j);
#pragma unroll
          for (int i = 0; i < L; ++i) read_x(o, x, i);
        }
        // every wave has read its first operands before their buffer is loaded again
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        // (one loop: a second one for the last steps had the accumulators in other registers, and copies between)
#pragma nounroll
        for (int p = 0; p < P; ++p) {
          if (p + 3 == P && more) aim_matrix(tn);
          if (p + kXBufs == P && more) aim_rows();
          step(p, p + 3 < P || more);
        }
      }
    };
    if (kRuns >= 6 && live == 6) run(std::integral_constant<int, kRuns >= 6 ? 6 : 0>{});
    else if (kRuns >= 5 && live == 5) run(std::integral_constant<int, kRuns >= 5 ? 5 : 0>{});
    else if (kRuns >= 4 && live == 4) run(std::integral_constant<int, kRuns >= 4 ? 4 : 0>{});
    else if (kRuns >= 3 && live == 3) run(std::integral_constant<int, kRuns >= 3 ? 3 : 0>{});
    else if (live == 2) run(std::integral_constant<int, 2>{});
    else if (live == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 0>{});
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
      if (i < live) {
        const int m = kRun * (run0 + i) + r;
        if (a.ydtype == 1) f8_store_bf16(a, acc[i], t.s0 + m, m < t.M, t.n0 + 64 * wn);
        else f8_store_f32(a, acc[i], t.s0 + m, m < t.M, t.n0 + 64 * wn);
      }
    if (!more) break;
    next = deal.answer(next);
    t = tn;
  }
}

}  // namespace

// Results in bf16 come from the 8-bit cores, which cut each of a block's products 13 bits below the largest one's binade (f8.h: the
// bound, what it does to a row, and what exact sums cost); so do the float32 parts of a token's sum that is rounded to bf16. Results in
// float32 take bf16 cores and keep all bits of every product (EXACT).
// Offsets within the rows and within one matrix are 32 bits wide.
bool f8_tiles_can(const F8Args& a) {
  const long long rows = a.perm ? a.T : a.A, stored = a.back ? a.K : a.N;
  return rows * a.xb * kF8Block < (1LL << 32) && stored * a.wb * kF8Block < (1LL << 32);
}

// Strips of 256 results a row, or of 128 where those would leave CUs without a tile. Measured, 128 against 256: one matrix
// [1024, 2048], 128 rows 13.6 us against 19.6, 2,048 14.9 against 20.7, 8,192 (256 tiles of 256) 28 against 25; the
// turned one, 2,048 rows 12.4 against 14.9, 8,192 (512 tiles) 36 against 28; experts [2048, 512] of 16 tokens 49 against 37.
// Tiles of 192 rows, whose rows have two buffers, where groups have more than 112 on average. Groups of one size, 192 against
// 128: [1024, 2048] 112 rows 33.5 us against 33.5, 144 35.4 against 40.5, 192 39.7 against 45.2, 256 53.4 against 51.8, 384 68
// against 73; experts of 8,192 tokens (176 rows) 320 against 358, of 4,096 (88 rows) 263 against 246. One matrix has no use for
// them: 8,192 rows of [1024, 2048] 31.9 against 25.4, where tiles of 128 fill the CUs once.
// Tiles are dealt to the workgroups in turn, or, of a turned matrix, taken from counters, which a launch before clears: where a
// group's strips are many, its steps too, and its rows few. Measured, taken against dealt: turned [1024, 2048] (8 strips, 8 steps),
// 1,024 tokens 218 us against 231, 8,192 (176 rows a group) 355 against 347, [512, 1024] (4 strips, 4 steps), 1,024 tokens 69
// against 67, [768, 4096] 185 against 194. Not turned no case gained: [2048, 1024], 1,024 tokens 227 against 224; [1024, 2048], 8,192 331
// against 314, 256 unevenly loaded 53 against 45.
hipError_t launch_f8_tiles(F8Args a, hipStream_t s) {
  const int cap = device_cus();
  const int strip = mx4_row_tiles(a) * ((a.N + 255) / 256) < cap ? 128 : 256;
  const long long groups = a.offsets ? (a.A < a.E_tot ? a.A : a.E_tot) : 1, strips = (a.N + strip - 1) / strip;
  const bool tall = strip == 256 && a.offsets && a.A > 112 * groups;
  const int tm = tall ? 192 : 128;
  const long long most = ((long long)(a.A + tm - 1) / tm + (a.offsets ? a.E_tot : 0)) * strips;
  const dim3 g((unsigned)(most < cap ? most : cap));
  if (most <= cap || g.x % kXcds || strips < 8 || a.xb < 6 || a.A > 96 * groups) a.counter = nullptr;
  if (a.counter) launch_mx4_zero(a.counter, s);
#define TILES(BACK, EXACT, NAME) \
  if (tall) MOE_LAUNCH(NAME "_192", s, (f8_tiles<BACK, EXACT, 4, 192>), g, dim3(kThreads), 0, s, a); \
  else if (strip == 256) MOE_LAUNCH(NAME, s, (f8_tiles<BACK, EXACT, 4, 128>), g, dim3(kThreads), 0, s, a); \
  else MOE_LAUNCH(NAME "_strip128", s, (f8_tiles<BACK, EXACT, 2, 128>), g, dim3(kThreads), 0, s, a)
  if (a.back && a.exact) { TILES(true, true, "f8_tiles_back"); }
  else if (a.back) { TILES(true, false, "f8_tiles_back"); }
  else if (a.exact) { TILES(false, true, "f8_tiles"); }
  else { TILES(false, false, "f8_tiles"); }
#undef TILES
  return hipGetLastError();
}

}  // namespace moe
