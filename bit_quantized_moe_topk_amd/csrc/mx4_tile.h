// What the tile kernels of the microscaled products share: how a launch's rows
// are dealt to tiles, direct loads into LDS, the layout of row tiles there, and
// how results are stored (header-only).
//
// A group's rows are dealt to its tiles in whole runs of 32, evenly (160 rows:
// 96 and 64, not 128 and 32): a run that is not there costs no products, and
// what a tile costs whatever its rows is spread over as many products as there are.
#pragma once

#include "mx4.h"
#include "sched.h"

namespace moe {

constexpr int kTM = 128;   // rows per tile, at most

// Stage layout in LDS: rows of 64 bf16 values, the eight 16-byte chunks of row m at
// positions q ^ ((m >> 1) & 7): the 16 rows that a quarter of a wave's fragment
// read takes then hit all 64 banks once.
__device__ inline int chunk_at(int m, int q) { return m * 8 + (q ^ ((m >> 1) & 7)); }

struct TileInfo {
  int e, s0, M, n0;
};

// Tiles of a launch: base[e] = the tiles before group e (of one strip of matrix
// rows). 16 bits hold them: 2^22 rows in tiles of 128 make 32,768, and one more
// a group. Tiles of 16 rows are for groups of up to kFewRowsF32 rows on average.
template <int CAP>
struct TilesOf {
  uint16_t base[CAP];
};
constexpr int kMaxTiles = 65535;
constexpr int kFewRowsF32 = 80;  // (what was measured: mx4_rows.hip)
static_assert(kMx4MaxRows / kTM + MOE_MAX_E_DEV + 1 <= kMaxTiles, "tiles of 128 rows");
static_assert((MOE_MAX_E_DEV + 1) * (kFewRowsF32 / 16 + 1) <= kMaxTiles, "tiles of 16 rows");
typedef TilesOf<MOE_MAX_E_DEV + 4> Tiles;

// Memory that tiles_init needs besides, free afterwards (past a barrier).
struct TilesScratch {
  int first[MOE_MAX_E_DEV + 4];  // first row of each group, and the end
  int wsum[16];
};

template <int TM = kTM, int CAP>
__device__ inline int tiles_init(TilesOf<CAP>& t, TilesScratch& w, const Mx4Args& a) {
  if (!a.offsets) return (a.A + TM - 1) / TM;
  constexpr int kAtOnce = 8;  // offsets on their way per thread
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int e0 = tid; e0 <= a.E_tot; e0 += kAtOnce * nt) {
    int v[kAtOnce];
#pragma unroll
    for (int z = 0; z < kAtOnce; ++z) v[z] = a.offsets[min(e0 + z * nt, a.E_tot)];
#pragma unroll
    for (int z = 0; z < kAtOnce; ++z)
      if (e0 + z * nt <= a.E_tot) w.first[e0 + z * nt] = cut_offset(a, v[z]);
  }
  __syncthreads();
  // this thread's groups are neighbours: their tiles, the sum of all before, and the places
  const int per = (a.E_tot + nt - 1) / nt, lo = min(a.E_tot, tid * per), hi = min(a.E_tot, lo + per);
  int n = 0;
  for (int e = lo; e < hi; ++e) n += max(0, w.first[e + 1] - w.first[e] + TM - 1) / TM;
  const int incl = wave_inclusive_scan(n);
  if ((tid & 63) == 63) w.wsum[tid >> 6] = incl;
  __syncthreads();
  int at = incl - n, all = 0;
  for (int i = 0; i < nt >> 6; ++i) {
    if (i < tid >> 6) at += w.wsum[i];
    all += w.wsum[i];
  }
  for (int e = lo; e < hi; ++e) {
    t.base[e] = (uint16_t)min(at, kMaxTiles);
    at += max(0, w.first[e + 1] - w.first[e] + TM - 1) / TM;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(min(all, kMaxTiles));  // more only where groups overlap, as they must not
}

// The last group whose first tile is at most ti.
template <int CAP>
__device__ inline int tile_group(const TilesOf<CAP>& t, int E_tot, int ti) {
  int lo = 0, hi = E_tot;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.base[mid] <= ti) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Item `id` of `items` (counted from the last group's end), strips of `strip` matrix rows; rows dealt in runs of RUN.
template <int TM = kTM, int RUN = 32, int CAP>
__device__ inline TileInfo tile_of(const TilesOf<CAP>& t, const Mx4Args& a, int id, int items, int strips, int strip) {
  TileInfo i;
  const int item = items - 1 - id, ti = item / strips;
  int r0 = 0, rows = a.A, of = (a.A + TM - 1) / TM, j = ti;
  i.e = 0;
  if (a.offsets) {
    i.e = __builtin_amdgcn_readfirstlane(tile_group(t, a.E_tot, ti));
    r0 = __builtin_amdgcn_readfirstlane(first_row(a, i.e));
    rows = __builtin_amdgcn_readfirstlane(first_row(a, i.e + 1)) - r0;
    j = ti - __builtin_amdgcn_readfirstlane((int)t.base[i.e]);
    of = (rows + TM - 1) / TM;
  }
  const int runs = (rows + RUN - 1) / RUN;
  const int a0 = (int)((long long)j * runs / of) * RUN, a1 = (int)((long long)(j + 1) * runs / of) * RUN;
  i.s0 = r0 + a0;
  i.M = min(a1, rows) - a0;
  i.n0 = (item - ti * strips) * strip;
  return i;
}

// The order in which workgroups take items, the last group's first (a shared
// expert's full tiles). Workgroup g runs on XCD g % 8, and runs of consecutive
// items go to one XCD, where they share rows or a matrix through its L2.
// Without counters every workgroup takes one item of each round. With them
// (kCounters, zeroed before the launch) it takes the next of its XCD's that
// nobody has, and when there is none another XCD's: tiles differ in cost by up
// to four, and whoever is dealt one more, or heavier ones, has the chip wait
// (the gradient of 1,024 tokens: 237 us dealt, 200 taken). An item is asked for
// a whole item before it is needed, so nobody waits for the answer but at the end.
constexpr int kXcds = 8, kCounters = kXcds;  // counters 32 words apart

struct Deal {
  int items, G;
  uint32_t* counter;
  int* slot;     // LDS
  uint32_t asked;

  __device__ int run() const { return G / kXcds; }  // items of a round on one XCD
  __device__ int item_of(int xcd, uint32_t q) const {
    const long long i = ((long long)(q / run()) * kXcds + xcd) * run() + q % run();
    return i < items ? (int)i : 0x7FFFFFFF;
  }
  __device__ int first() const { return G % kXcds ? blockIdx.x : item_of(blockIdx.x % kXcds, blockIdx.x / kXcds); }
  __device__ uint32_t take(int xcd) {
    return run() + __hip_atomic_fetch_add(counter + 32 * xcd, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ void ask() {
    if (counter && threadIdx.x == 0) asked = take(blockIdx.x % kXcds);
  }
  // The item after `next`, by all threads. (Another tile's barriers lie before the next write to the slot.)
  __device__ int answer(int next) {
    if (!counter) return next < items ? next + G : next;
    if (threadIdx.x == 0) {
      int xcd = blockIdx.x % kXcds, i = item_of(xcd, asked);
      for (int z = 1; z < kXcds && i >= items; ++z) {
        xcd = xcd + 1 == kXcds ? 0 : xcd + 1;
        i = item_of(xcd, take(xcd));
      }
      *slot = i;
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    return __builtin_amdgcn_readfirstlane(*reinterpret_cast<volatile int*>(slot));
  }
};

__device__ inline uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}

// Direct loads as instructions of their own: lane l's bytes land at LDS
// address `to` + 16 l (4 l). The compiler would make every LDS read wait for
// all of them; here step_done() is the one wait, at the end of a step. (m0 has
// no other user in these kernels.)
__device__ inline void stream16(const void* base, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(__builtin_amdgcn_readfirstlane(to)), "v"(off), "s"(base) : "memory");
}
__device__ inline void stream4(const void* base, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               :: "s"(__builtin_amdgcn_readfirstlane(to)), "v"(off), "s"(base) : "memory");
}
__device__ inline void stream16(const void* src, uint32_t to) {  // an address of each lane's own
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(__builtin_amdgcn_readfirstlane(to)), "v"(src) : "memory");
}
__device__ inline void stream4(const void* src, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :: "s"(__builtin_amdgcn_readfirstlane(to)), "v"(src) : "memory");
}
// This wave's direct loads have landed and its LDS reads are done; then the same for every wave.
// (IN_FLIGHT: all but the last so many).
template <int IN_FLIGHT = 0>
__device__ inline void step_done() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(IN_FLIGHT) : "memory");
}

// Stores one run of 32 rows: acc[j][v] is matrix row n0 + 32 j + 8 (v / 4) +
// 4 h + v % 4, row s0 + r. For 16-bit results the lane halves swap quads, so
// that each lane holds eight neighbours (h 0: of an even quad pair, h 1: of
// the odd one) and stores 16 bytes.
__device__ inline uint32_t pack_bf16(float a, float b) {
  typedef float float2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t{a, b}), bf16x2_t));
}

__device__ inline void store_run(const Mx4Args& a, const floatx16_t (&acc)[2], int s0, int M, int n0) {
  const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
  if (a.ydtype == 1) {
    uint16_t* y = static_cast<uint16_t*>(a.y) + (size_t)(s0 + r) * a.N;
    const bool wide = a.N % 8 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        uint32_t p[4];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const auto s = __builtin_amdgcn_permlane32_swap(pack_bf16(acc[j][4 * q + 2 * z], acc[j][4 * q + 2 * z + 1]),
                                                          pack_bf16(acc[j][4 * q + 2 * z + 4], acc[j][4 * q + 2 * z + 5]),
                                                          false, false);
          p[z] = s[0];
          p[2 + z] = s[1];
        }
        const int n = n0 + 32 * j + 8 * (q + h);
        if (r < M) {
          if (wide) {
            if (n < a.N) *reinterpret_cast<uint4*>(y + n) = make_uint4(p[0], p[1], p[2], p[3]);
          } else {
#pragma unroll
            for (int z = 0; z < 8; ++z)
              if (n + z < a.N) y[n + z] = (uint16_t)(p[z / 2] >> (16 * (z & 1)));
          }
        }
      }
  } else if (r < M) {
    float* y = static_cast<float*>(a.y) + (size_t)(s0 + r) * a.N;
    const bool wide = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + 32 * j + 8 * q + 4 * h;
        if (wide) {
          if (n < a.N)
            *reinterpret_cast<float4*>(y + n) =
                make_float4(acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]);
        } else {
#pragma unroll
          for (int z = 0; z < 4; ++z)
            if (n + z < a.N) y[n + z] = acc[j][4 * q + z];
        }
      }
  }
}

}  // namespace moe
