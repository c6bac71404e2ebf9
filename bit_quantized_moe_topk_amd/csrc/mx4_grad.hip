// Gradients of many rows through a microscaled matrix, dx = dy W, on 16x16x32
// matrix-core tiles.
//
// The sum runs along the matrix's rows while its blocks lie along the columns.
// No transposed copy is needed: a lane takes one dword of codes, eight
// neighbouring columns, from each of the eight matrix rows that its part of a
// product step covers, converts each with its own scale, and regroups pairs of
// rows (mx4_columns): 32 conversions and 32 permutes give the operands of
// eight products, product c covering the columns 8 r + c. They serve up to
// four 16-row tiles.
//
// What bounds it where groups hold a few rows is bringing the matrices: 1,024
// tokens x 11, 512 experts, [1024, 2048] read 617 MB and write 93 MB in 192 us,
// 72 % of a copy's rate. With one workgroup a CU and a barrier a stage that
// leaves the waves waiting for 38 % of their time, while the vector units are
// busy for a third of it and the matrix cores for an eighth.
//
// A workgroup takes up to 128 rows by 128 WK columns: two waves down, WK
// across, 64 rows by 128 columns a wave, in stages of 64 matrix rows.
#include "mx4_tile.h"

namespace moe {
namespace {

constexpr int kGN = 64;  // matrix rows per stage

// The operands of eight products from eight matrix rows' code dwords and
// scales: w[c] holds column c of the eight rows.
__device__ inline void mx4_columns(const uint32_t (&code)[8], const float (&sc)[8], bf16x8_t (&w)[8]) {
  uint32_t p[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    p[j][0] = mx4_pair<0>(code[j], sc[j]);
    p[j][1] = mx4_pair<1>(code[j], sc[j]);
    p[j][2] = mx4_pair<2>(code[j], sc[j]);
    p[j][3] = mx4_pair<3>(code[j], sc[j]);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    auto two = [&](int j) {
      return c & 1 ? hi_pair(p[j][c / 2], p[j + 1][c / 2]) : lo_pair(p[j][c / 2], p[j + 1][c / 2]);
    };
    w[c] = __builtin_bit_cast(bf16x8_t, make_uint4(two(0), two(2), two(4), two(6)));
  }
}

template <int P, int WK>
struct GradBuf {
  uint4 d[P][kTM * 8];         // dy's rows (chunk_at)
  uint4 w[kGN * 4 * WK];       // matrix rows: 4 WK blocks each (code_at)
  uint8_t s[kGN * 4 * WK];     // its 4 WK scales
};

// Position of chunk c (a block of codes) of matrix row n: the four rows 8 g + j
// that one read of a wave takes lie on different quarters of the banks.
template <int WK>
__device__ inline int code_at(int n, int c) {
  return n * 4 * WK + (c ^ (4 * ((n >> 3) & (WK - 1))));
}

// STREAM: dy bf16, its rows readable 16 bytes at a time, N a multiple of 64,
// scales readable four at a time: everything comes by direct loads, two stages
// ahead in three buffers. Else through registers into the other of two buffers:
// a stage's loads are waited for before the last one's products, not under them.
// The loads run on across tiles.
template <int P, int WK, bool STREAM>
__global__ __launch_bounds__(128 * WK, P == 1 ? 2 : 1) void tiles_gradient(Mx4Args a, bool vec) {
  constexpr int kBufs = STREAM ? 3 : 2, kThreads = 128 * WK;
  constexpr int kDL = 16 / (2 * WK), kWL = kGN * 4 * WK / 64 / (2 * WK);  // direct loads a wave and stage
  __shared__ GradBuf<P, WK> buf[kBufs];
  __shared__ Tiles tiles;
  __shared__ floatx4_t meet[2 * WK][4][64];
  constexpr int strip = 128 * WK;
  const int strips = (a.K + strip - 1) / strip;
  const int items = tiles_init(tiles, *reinterpret_cast<TilesScratch*>(buf), a) * strips;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4, wk = wave % WK, wm = wave / WK;
  const int nb = mx4_blocks(a.K), S = (a.N + kGN - 1) / kGN;
  __shared__ int slot;
  Deal deal{items, (int)gridDim.x, a.counter, &slot, 0u};
  int item = deal.first();
  if (item >= items) return;
  deal.ask();
  int next = deal.answer(item);
  // load cursor: stage ls of tile lt, into buffer lb; `next` is the item that it goes to then
  TileInfo lt = tile_of(tiles, a, item, items, strips, strip);  // n0: its first column
  int ls = 0, lb = 0;
  bool crossed = false;  // it is in the next item
  bool rows = false;  // whether this wave's last load() brought rows of dy
  int held = 0;       // stages loaded and not used yet
  // the next stage, of whatever tile it is, if there is one
  auto load = [&]() __attribute__((always_inline)) {
    if (ls == S) {
      if (crossed || next >= items) return;
      crossed = true;
      lt = tile_of(tiles, a, next, items, strips, strip);
      ls = 0;
    }
    ++held;
    const int s = ls++, b0 = lt.n0 / 32;
    const char* wbase = reinterpret_cast<const char*>(a.wc) + (size_t)lt.e * a.N * nb * 16;
    const uint8_t* sbase = a.ws + (size_t)lt.e * a.N * nb;
    GradBuf<P, WK>& B = buf[lb];
    lb = lb + 1 == kBufs ? 0 : lb + 1;
    rows = 8 * kDL * wave < ((lt.M + 15) & ~15);
    if constexpr (STREAM) {
#pragma unroll
      for (int u = 0; u < kDL; ++u) {
        if (!rows) break;
        const int m = 8 * (kDL * wave + u) + (lane >> 3);
        const int row = lt.s0 + min(m, lt.M - 1);
        stream16(static_cast<const char*>(a.x) + s * 2 * kGN,
                 (uint32_t)row * (uint32_t)(2 * a.ldx) + 16 * ((lane & 7) ^ ((m >> 1) & 7)),
                 lds_offset(B.d[0]) + 1024 * (kDL * wave + u));
      }
#pragma unroll
      for (int u = 0; u < kWL; ++u) {
        const int at = 64 * (kWL * wave + u) + lane, n = at / (4 * WK);
        const int c = (at % (4 * WK)) ^ (4 * ((n >> 3) & (WK - 1)));
        stream16(wbase, (uint32_t)(s * kGN + n) * (uint32_t)(16 * nb) + 16 * min(b0 + c, nb - 1),
                 lds_offset(B.w) + 1024 * (kWL * wave + u));
      }
      if (lane < 32) {
        const int at = 32 * wave + lane, n = at / WK, z = at % WK;
        stream4(sbase, (uint32_t)(s * kGN + n) * nb + min(b0 + 4 * z, nb - 4), lds_offset(B.s) + 128 * wave);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kTM * 8 / kThreads; ++i) {
        const int at = i * kThreads + tid, m = at / 8, q = at % 8, n = s * kGN + 8 * q;
        const size_t row = (size_t)(lt.s0 + m) * a.ldx;
        const bool there = m < lt.M && n < a.N;
        if constexpr (P == 1) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (there) v = load8_bf16(static_cast<const uint16_t*>(a.x) + row, n, a.N, vec);
          B.d[0][chunk_at(m, q)] = v;
        } else {
          float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (there) load8_f32(static_cast<const float*>(a.x) + row, n, a.N, vec, f);
          split3x8(f, B.d[0][chunk_at(m, q)], B.d[P > 1 ? 1 : 0][chunk_at(m, q)], B.d[P > 1 ? 2 : 0][chunk_at(m, q)]);
        }
      }
      // matrix rows past N: scales of 2^-127, zeros in dy
#pragma unroll
      for (int i = 0; i < kGN * 4 * WK / kThreads; ++i) {
        const int at = i * kThreads + tid, n = at / (4 * WK), c = at % (4 * WK);
        const size_t blk = (size_t)min(s * kGN + n, a.N - 1) * nb + min(b0 + c, nb - 1);
        B.w[code_at<WK>(n, c)] = *reinterpret_cast<const uint4*>(wbase + 16 * blk);
        B.s[at] = s * kGN + n < a.N ? sbase[blk] : 0;
      }
    }
  };
  load();
  if (STREAM) load();
  // The next stage has landed; a load() beyond it may be in flight (there is none where a tile is one stage and the
  // item after the next is not known yet).
  auto done = [&]() __attribute__((always_inline)) {
    if (!STREAM || held < 2) step_done();
    else if (rows) step_done<kDL + kWL + 1>();
    else step_done<kWL + 1>();
  };
  done();
  int cb = 0;  // the buffer whose turn it is
  while (item < items) {
    deal.ask();
    const TileInfo t = tile_of(tiles, a, item, items, strips, strip);
    // Up to 64 rows: both waves take all of them, each half of every stage's matrix rows, so that
    // the weights are converted once; their sums meet at the end. More: half of the rows each.
    const int U = (t.M + 15) / 16;
    const bool shared = U <= 4;
    const int u0 = wm && !shared ? (U + 1) / 2 : 0, live = shared ? U : wm ? U / 2 : (U + 1) / 2;
    floatx4_t acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[i][c] = floatx4_t{};
    auto run = [&](auto LL, auto SH) __attribute__((always_inline)) {
      constexpr int L = decltype(LL)::value;
      constexpr bool kShared = decltype(SH)::value;
      for (int s = 0; s < S; ++s) {
        load();
        {
          const GradBuf<P, WK>& B = buf[cb];
#pragma unroll
          for (int z = 0; z < (kShared ? 1 : 2); ++z) {
            const int half = kShared ? wm : z;
            uint32_t code[8];
            float sc[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int n = 32 * half + 8 * g + j;
              code[j] = reinterpret_cast<const uint32_t*>(B.w)[4 * code_at<WK>(n, 4 * wk + (r >> 2)) + (r & 3)];
              sc[j] = mx4_scale(B.s[n * 4 * WK + 4 * wk + (r >> 2)]);
            }
            bf16x8_t w[8];
            mx4_columns(code, sc, w);
#pragma unroll
            for (int p = P - 1; p >= 0; --p)
#pragma unroll
              for (int i = 0; i < L; ++i) {
                const bf16x8_t d = __builtin_bit_cast(bf16x8_t, B.d[p][chunk_at(16 * (u0 + i) + r, 4 * half + g)]);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  acc[i][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(d, w[c], acc[i][c], 0, 0, 0);
              }
          }
        }
        --held;
        done();
        cb = cb + 1 == kBufs ? 0 : cb + 1;
      }
    };
    if (shared) {
      if (live == 4) run(std::integral_constant<int, 4>{}, std::true_type{});
      else if (live == 3) run(std::integral_constant<int, 3>{}, std::true_type{});
      else if (live == 2) run(std::integral_constant<int, 2>{}, std::true_type{});
      else run(std::integral_constant<int, 1>{}, std::true_type{});
      // of two 16-row tiles the first wave finishes the even one and the second the odd one; each
      // gives the other its sums, four columns of eight at a time
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        if (i >= live) break;
#pragma unroll
        for (int c0 = 0; c0 < 8; c0 += 4) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // (branches, not indexes: accumulators stay in registers)
            if (wm) meet[wave][c][lane] = acc[i][c0 + c];
            else meet[wave][c][lane] = acc[i + 1][c0 + c];
          }
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const floatx4_t o = meet[wave ^ WK][c][lane];
            if (wm) acc[i + 1][c0 + c] += o;
            else acc[i][c0 + c] += o;
          }
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
      }
    } else {
      if (live == 4) run(std::integral_constant<int, 4>{}, std::false_type{});
      else if (live == 3) run(std::integral_constant<int, 3>{}, std::false_type{});
      else run(std::integral_constant<int, 2>{}, std::false_type{});
    }
    // acc[i][c][v]: row 16 (u0 + i) + 4 g + v, column k + c: eight neighbours a lane
    const int k = t.n0 + 128 * wk + 8 * r;
    const bool wide = a.K % 8 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= live || (shared && (i & 1) != wm)) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int m = 16 * (u0 + i) + 4 * g + v;
        if (m >= t.M || k >= a.K) continue;
        const size_t at = (size_t)(t.s0 + m) * a.K + k;
        if (a.ydtype == 1) {
          uint16_t* y = static_cast<uint16_t*>(a.y) + at;
          const uint4 o = make_uint4(pack_bf16(acc[i][0][v], acc[i][1][v]), pack_bf16(acc[i][2][v], acc[i][3][v]),
                                     pack_bf16(acc[i][4][v], acc[i][5][v]), pack_bf16(acc[i][6][v], acc[i][7][v]));
          if (wide) {
            *reinterpret_cast<uint4*>(y) = o;
          } else {
            const uint32_t p[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (k + c < a.K) y[c] = (uint16_t)(p[c / 2] >> (16 * (c & 1)));
          }
        } else {
          float* y = static_cast<float*>(a.y) + at;
          if (wide) {
            reinterpret_cast<float4*>(y)[0] = make_float4(acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]);
            reinterpret_cast<float4*>(y)[1] = make_float4(acc[i][4][v], acc[i][5][v], acc[i][6][v], acc[i][7][v]);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (k + c < a.K) y[c] = acc[i][c][v];
          }
        }
      }
    }
    item = next;
    crossed = false;
    if (item < items) next = deal.answer(item);
  }
}

}  // namespace

hipError_t launch_mx4_grad_tiles(Mx4Args a, hipStream_t s) {
  const int nb = mx4_blocks(a.K);
  const bool vec = rows_vec(a.x, a.ldx, a.xdtype == 1 ? 2 : 4);
  const bool stream = a.xdtype == 1 && vec && a.N % kGN == 0 && nb % 4 == 0 &&
                      (reinterpret_cast<uintptr_t>(a.ws) & 3) == 0 && 16LL * a.N * nb < (1LL << 32) &&
                      a.A * a.ldx * 2 < (1LL << 32);
  const int strip = stream ? 512 : 256;
  const long long strips = (a.K + strip - 1) / strip;
  const long long most = ((long long)(a.A + kTM - 1) / kTM + (a.offsets ? a.E_tot : 0)) * strips;
  const int cap = (stream || a.xdtype == 0 ? 1 : 2) * device_cus();
  const dim3 g((unsigned)(most < cap ? most : cap));
  if (most <= cap || g.x % kXcds) a.counter = nullptr;
  else if (a.counter) launch_mx4_zero(a.counter, s);
  if (stream) MOE_LAUNCH("mx4_grad_stream", s, (tiles_gradient<1, 4, true>), g, dim3(512), 0, s, a, vec);
  else if (a.xdtype == 1) MOE_LAUNCH("mx4_grad_tiles", s, (tiles_gradient<1, 2, false>), g, dim3(256), 0, s, a, vec);
  else MOE_LAUNCH("mx4_grad_tiles", s, (tiles_gradient<3, 2, false>), g, dim3(256), 0, s, a, vec);
  return hipGetLastError();
}

}  // namespace moe
