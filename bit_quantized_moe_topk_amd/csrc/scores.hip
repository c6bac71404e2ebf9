// Routing by scores: sigmoid or softmax scores, a bias that takes part in the
// selection alone, groups of experts, top-k and gates, and the gates' gradient
// for the logits.
//
// One wave a token, expert lane + 64 i in slot i. The order is that of values in
// 64 bits (score + bias): in 32, two experts a last place apart would come in the
// order of their roundings. But 64 bits for all 512 experts of 8,192 tokens took 55 us.
// So scores are computed in 32 first, which with a bias are off by less than a
// margin; what is not within it of a border is settled:
//   groups  : their values in 32 bits, unless the last that stays and the first that
//             goes are near each other; then those of each group's best two in 64.
//   experts : all within the margin of a lower bound of the k-th (topk.h's threshold)
//             are candidates, one a lane, ranked by counting; where two of them are near
//             each other, by their values in 64 bits, which take all lanes at once. Without a
//             bias the logits are the order.
// What remains (over 64 candidates or ranks; a third expert of a group near its
// second where groups are near) goes through 64 bits for all experts and k rounds.
//
// Measured: 8,192 tokens of 512 experts in 8 groups, k 8, with a bias 21.5 us, and 7.2 its gradient (64 bits
// throughout: 55 and 8.2); a window of 4 tokens 6.9, one chain of dependent steps. Bound by vector instructions, 1,060 a
// token, which have the vector units busy half of the time, and the steps that wait for one another; its 17 MB would take 3.4.
// From k of about 40 of 512 experts on there are more than 64 candidates, and from 65 on always: 64 bits for all, k rounds
// (one group: k 32 28 us, 40 84, 64 195, 100 323; its gradient 11, 12, 15, 30, past 64 an assignment after the other). Of 1,000 tokens x 100
// experts all that stay are candidates, which rank one another in turn: 10.8 us.
// Exponentials by the instruction (score_near) only screen. Gates are of expf and of sums in 32 bits: within (E + 8) 2^-24 of
// their value, and of a softmax |l - largest| 2^-24 besides, the rounding of that difference.
#include "gemv.h"
#include "norm.h"
#include "topk.h"

namespace moe {
namespace {

// Order-preserving code of a double: NaN is 1, below -inf; 0 marks what cannot be selected.
__device__ inline uint64_t orderable64(double v) {
  if (v != v) return 1ull;
  const uint64_t u = __double_as_longlong(v == 0.0 ? 0.0 : v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
constexpr uint64_t kOff = 0x000FFFFFFFFFFFFFull;  // -inf's code
constexpr uint32_t kOff32 = 0x007FFFFFu;          // and the one of orderable()
__device__ inline double from_orderable64(uint64_t o) {
  return __longlong_as_double((o >> 63) ? (o & 0x7FFFFFFFFFFFFFFFull) : ~o);
}

__device__ inline double wave_sum64(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ inline float wave_maxf(float v) { return from_orderable(wave_reduce<true>(orderable(v))); }

__device__ inline float logit_at(const ScoreArgs& a, int t, int e) {
  const size_t at = (size_t)t * a.ld + e;
  return a.bf16 ? bf16_lo(static_cast<const uint16_t*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
}

// What a softmax needs of its row: the largest logit (NaN of a row with a NaN, -inf of one that is all off) and
// the sum of exponentials (1 where only their ratios matter).
struct Base {
  float top;
  double total;
};
__device__ inline double score64(const ScoreArgs& a, const Base& b, float l) {
  if (!a.softmax) return 1.0 / (1.0 + exp(-(double)l));
  return b.top == -INFINITY ? 0.0 : exp((double)l - (double)b.top) / b.total;
}
// The same in 32 bits, within 2^-21, of a softmax over 2,048 experts 2^-19.6 of its share (the total's roundings), and
// of a sigmoid relative to its value, down to 2^-126.
__device__ inline float score32(const ScoreArgs& a, const Base& b, float l) {
  if (!a.softmax) return __builtin_amdgcn_rcpf(1.f + expf(-l));
  return b.top == -INFINITY ? 0.f : expf(l - b.top) * __builtin_amdgcn_rcpf((float)b.total);
}

// What a biased score is screened by: as near as score32, but not relative to small ones. (Two shares are at most 1 together,
// so a group's margin, and a candidate's, of 2^-18 holds their errors.)
__device__ inline float score_near(const ScoreArgs& a, const Base& b, float l) {
  if (!a.softmax) return __builtin_amdgcn_rcpf(1.f + __expf(-l));
  return b.top == -INFINITY ? 0.f : __expf(l - b.top) * __builtin_amdgcn_rcpf((float)b.total);
}

constexpr int kWaves = 4;  // tokens per workgroup

template <int P>
struct Scratch {
  union {
    uint64_t key[64 * P];  // 64 bits for all experts
    struct {
      float l[64 * P];  // the row's logits
      float c[64 * P];  // what ranks an expert within its group
    };
  };
  uint2 cand[64];  // candidates: what ranks them, and which
};

// The sum of a row's exponentials in 64 bits.
template <int P>
__device__ inline double total64(const Scratch<P>& sc, int E, float top) {
  double v = 0.0;
#pragma unroll 1
  for (int e = threadIdx.x & 63; e < E; e += 64) v += top == -INFINITY ? 0.0 : exp((double)sc.l[e] - (double)top);
  return wave_sum64(v);
}

__device__ inline uint32_t from_lane(uint32_t v, int j) { return __builtin_amdgcn_readlane(v, j); }
__device__ inline uint64_t from_lane(uint64_t v, int j) {
  return (uint64_t)from_lane((uint32_t)(v >> 32), j) << 32 | from_lane((uint32_t)v, j);
}

// Group g's value (an order code) lies in lanes g * per and on: whether this lane's is among the `keep` largest, equal ones
// in favour of the lower group; the bits of all lanes.
template <typename V>
__device__ inline uint64_t kept_groups(const ScoreArgs& a, V v, int per, bool* stays) {
  const int lane = threadIdx.x & 63;
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) {
    const V o = from_lane(v, g * per);
    rank += o > v || (o == v && g * per < lane - lane % per);
  }
  *stays = lane / per < a.groups && rank < a.keep;
  return __ballot(*stays);
}

// The partner of a lane in the step o of a reduction over 2 o lanes that alone are equal within o.
__device__ inline uint32_t partner(uint32_t v, int o) {
  switch (o) {
    case 1: return dpp(v, 0xB1);
    case 2: return dpp(v, 0x4E);
    case 4: return dpp(v, 0x141);
    case 8: return dpp(v, 0x140);
    default: return __shfl_xor(v, o, 64);
  }
}
__device__ inline float partner(float v, int o) { return __uint_as_float(partner(__float_as_uint(v), o)); }

// 64 bits for all experts: groups by scanning them, then k rounds.
template <int P>
__device__ inline void select64(const ScoreArgs& a, int t, Base base, Scratch<P>& sc) {
  const int lane = threadIdx.x & 63;
  if (a.softmax) base.total = total64<P>(sc, a.E, base.top);
  uint64_t key[P];
  float l[P];
#pragma unroll
  for (int i = 0; i < P; ++i) l[i] = sc.l[lane + 64 * i];
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const double c = l[i] == -INFINITY ? -INFINITY : a.bias ? score64(a, base, l[i]) + (double)a.bias[min(lane + 64 * i, a.E - 1)] : (double)l[i];
    key[i] = lane + 64 * i < a.E ? orderable64(c) : 0ull;
    sc.key[lane + 64 * i] = key[i];
  }
  __builtin_amdgcn_wave_barrier();
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    uint64_t mine = 0;
    if (lane < a.groups) {
      uint64_t k1 = kOff, k2 = kOff;  // what is not above -inf is left out
      for (int e = lane * size; e < (lane + 1) * size; ++e) {
        const uint64_t k = sc.key[e];
        k2 = k > k1 ? k1 : k > k2 ? k : k2;
        k1 = k > k1 ? k : k1;
      }
      mine = k1;
      if (a.group_top == 2 && k1 > kOff) {
        double v1 = from_orderable64(k1), v2 = k2 == kOff ? 0.0 : from_orderable64(k2);
        if (!a.bias) {
          v1 = score64(a, base, (float)v1);
          if (k2 != kOff) v2 = score64(a, base, (float)v2);
        }
        mine = orderable64(v1 + v2);
      }
    }
    bool stays;
    const uint64_t kept = kept_groups(a, mine, 1, &stays);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 64 * i < a.E && !(kept >> ((lane + 64 * i) / size) & 1)) key[i] = 0ull;
  }
  double sum = 0.0;
  int mine = 0;
  float logit = 0.f;  // of rank `lane`
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = key[0];
    int e = lane;
    float x = l[0];
#pragma unroll
    for (int i = 1; i < P; ++i)
      if (key[i] > best) {
        best = key[i];
        e = lane + 64 * i;
        x = l[i];
      }
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t ob = __shfl_xor(best, o, 64);
      const int oe = __shfl_xor(e, o, 64);
      const float ox = __shfl_xor(x, o, 64);
      if (ob > best || (ob == best && oe < e)) {
        best = ob;
        e = oe;
        x = ox;
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 64 * i == e) key[i] = 0ull;
    if (lane == (j & 63)) mine = e;
    if (lane == j) logit = x;
    sum += score64(a, base, x);
    if ((j & 63) == 63 || j + 1 == a.k) {
      const int r = (j & ~63) + lane;
      if (r <= j) a.idx[(size_t)t * a.k + r] = mine;
    }
    if (j >= 64 && lane == 0) a.gates[(size_t)t * a.k + j] = x;  // its logit, until the sum is known
  }
  auto gate = [&](float x) {
    const double v = score64(a, base, x);
    return (float)((double)a.scale * (!a.renorm ? v : sum == 0.0 ? 0.0 : v / sum));
  };
  if (lane < a.k) a.gates[(size_t)t * a.k + lane] = gate(logit);
  for (int j = 64; j < a.k; ++j)  // (lane 0 reads what it wrote)
    if (lane == 0) a.gates[(size_t)t * a.k + j] = gate(a.gates[(size_t)t * a.k + j]);
}

// The three largest of a group's ranking values, the first two with their places.
struct Top3 {
  float v1, v2, v3;
  int e1, e2;
  __device__ void add(float v, int e) {
    const bool g1 = v > v1, g2 = v > v2;
    v3 = g2 ? v2 : fmaxf(v3, v);
    v2 = g1 ? v1 : g2 ? v : v2;
    e2 = g1 ? e1 : g2 ? e : e2;
    v1 = g1 ? v : v1;
    e1 = g1 ? e : e1;
  }
};

template <int P>
__global__ __launch_bounds__(64 * kWaves) void scores_forward(ScoreArgs a) {
  __shared__ Scratch<P> scratch[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  Scratch<P>& sc = scratch[wave];
  float l[P], bias[P];
  auto load = [&](int last) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < P; ++i) l[i] = logit_at(a, t, min(lane + 64 * i, last));
#pragma unroll
    for (int i = 0; i < P; ++i) bias[i] = a.bias ? a.bias[min(lane + 64 * i, last)] : 0.f;
  };
  if (a.E == 64 * P) load(64 * P - 1);  // (no limit to look at)
  else load(a.E - 1);
#pragma unroll
  for (int i = 0; i < P; ++i) sc.l[lane + 64 * i] = l[i];
  Base base{0.f, 1.0};
  if (a.softmax) {
    float top = -INFINITY;
    bool nan = false;  // (a maximum leaves it out)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      top = fmaxf(top, l[i]);
      nan |= l[i] != l[i];
    }
    top = wave_maxf(top);
    base.top = __any(nan) || top == INFINITY ? NAN : top;  // (such a row has no scores)
    if (a.bias || !a.renorm || base.top != base.top) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (lane + 64 * i < a.E) v += base.top == -INFINITY ? 0.f : expf(l[i] - base.top);
      base.total = wave_sum(v);
    }
  }
  // what ranks an expert: its logit, or score + bias in 32 bits
  float c[P];
#pragma unroll
  for (int i = 0; i < P; ++i) c[i] = l[i] == -INFINITY || !a.bias ? l[i] : score_near(a, base, l[i]) + bias[i];
  const int size = a.E / a.groups;
  uint64_t out = 0;  // bit i: slot i's group does not stay
  bool hard = a.k > 64;
  if (a.groups > 1 && a.keep < a.groups && !hard) {
#pragma unroll
    for (int i = 0; i < P; ++i) sc.c[lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    uint64_t kept;
    int per = 64;  // lanes a group, which share its experts
    while (per * a.groups > 64) per >>= 1;
    const int g = lane / per;
    Top3 top{-INFINITY, -INFINITY, -INFINITY, 0, 0};  // (what is not above -inf is left out, NaN too)
    if (g < a.groups)
      for (int e = g * size + lane % per; e < (g + 1) * size; e += per) top.add(sc.c[e], e);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      if (o >= per) continue;
      const Top3 u{partner(top.v1, o), partner(top.v2, o), partner(top.v3, o), (int)partner((uint32_t)top.e1, o),
                   (int)partner((uint32_t)top.e2, o)};
      top.add(u.v1, u.e1);
      top.add(u.v2, u.e2);
      top.v3 = fmaxf(top.v3, u.v3);
    }
    const bool ours = g < a.groups, live = top.v1 > -INFINITY, two = a.group_top == 2 && top.v2 > -INFINITY;
    float v = top.v1, margin = 0.f;
    if (a.bias || a.group_top == 2) {
      if (!a.bias) v = live ? score32(a, base, top.v1) : v;
      if (two) v += a.bias ? top.v2 : score32(a, base, top.v2);
      // (each term is rounded by itself: where they nearly cancel, by far more than the sum's own rounding)
      margin = a.bias ? 0x1p-18f + 0x1p-21f * (fabsf(top.v1) + (two ? fabsf(top.v2) : 0.f)) : fmaxf(0x1p-19f * v, 0x1p-126f);
    }
    bool stays;
    kept = kept_groups(a, orderable(v), per, &stays);
    // the least that stays and the most that goes
    const float lo = from_orderable(wave_reduce<false>(stays ? orderable(v) : 0xFFFFFFFFu));
    const float hi = wave_maxf(ours && !stays ? v : -INFINITY);
    const float most = wave_maxf(ours && live ? margin : 0.f);
    // (a sum past the range is -inf, as the value of a group that is off; its margin is infinite)
    const bool open = __any(ours && !stays && live);
    if (most > 0.f && open && !(most < INFINITY && lo - hi >= 2.f * most)) {
      // the best of a group in 32 bits need not be so in 64, where the next is near
      const float apart = 0x1p-17f + 0x1p-20f * fabsf(top.v2);
      hard = !(hi < INFINITY) || (a.bias && __any(ours && (a.group_top == 2 ? two && top.v3 > -INFINITY && !(top.v2 - top.v3 >= apart)
                                                                             : top.v2 > -INFINITY && !(top.v1 - top.v2 >= apart))));
      if (!hard) {
        Base exact = base;
        if (a.softmax && a.bias) exact.total = total64<P>(sc, a.E, base.top);
        double w = -INFINITY;
        if (ours && live) {
          w = a.bias ? score64(a, exact, sc.l[top.e1]) + (double)a.bias[top.e1] : score64(a, exact, top.v1);
          if (two) w += a.bias ? score64(a, exact, sc.l[top.e2]) + (double)a.bias[top.e2] : score64(a, exact, top.v2);
        }
        kept = kept_groups(a, ours ? orderable64(w) : (uint64_t)0, per, &stays);
      }
    }
    __builtin_amdgcn_wave_barrier();
    // a bit for each expert's group (exact: the quotient is under 64, and half an expert from a border)
    const float each = 1.f / (float)size;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int of = min((int)(((float)(lane + 64 * i) + 0.5f) * each), a.groups - 1);  // (a lane past the experts: any)
      out |= (kept >> (of * per) & 1 ? 0ull : 1ull) << i;
    }
  }
  uint32_t key[P], head = 0u;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < a.E && !(out >> i & 1) ? orderable(c[i]) : 0u;
    head = max(head, key[i]);
  }
  int n = 0;
  uint32_t least = 1u;  // candidates' least code: all that may be selected, where they are few
  if (!hard && a.keep * size > 64) {
    // the k-th largest of the lanes' largest, its last 13 bits open downward, a bit at a time
    least = 0u;
#pragma unroll
    for (int i = 31; i > 12; --i) {
      const uint32_t next = least | 1u << i;
      if (__popcll(__ballot(head >= next)) >= a.k) least = next;
    }
    least = max(least, 1u);
    if (a.bias && least > kOff32) {
      const float tau = from_orderable(least);
      least = orderable(tau - (0x1p-18f + 0x1p-21f * fabsf(tau)));
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) n += __popcll(__ballot(key[i] >= least));
  if (hard || n > 64) {
    select64<P>(a, t, base, sc);
    return;
  }
  int at = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const bool in = key[i] >= least;
    const uint64_t m = __ballot(in);
    if (in) {
      const int z = at + __popcll(m & lanemask_lt());
      sc.cand[z] = make_uint2(key[i], lane + 64 * i);
    }
    at += __popcll(m);
  }
  __builtin_amdgcn_wave_barrier();
  const bool in = lane < n;
  const uint32_t mine = in ? sc.cand[lane].x : 0u;
  const int e = in ? (int)sc.cand[lane].y : a.E;
  const float x = in ? sc.l[e] : 0.f;
  const float v = from_orderable(mine), apart = a.bias ? 0x1p-17f + 0x1p-20f * fabsf(v) : 0.f;
  int rank = 0;
  bool near = false;  // to another one: the order is open
  for (int j = 0; j < n; ++j) {
    const uint32_t o = from_lane(mine, j);
    const int oe = __builtin_amdgcn_readlane(e, j);
    rank += o > mine || (o == mine && oe < e);
    near |= oe != e && fabsf(from_orderable(o) - v) < apart;
  }
  float s = in ? a.softmax ? score32(a, base, x) : 1.f / (1.f + expf(-x)) : 0.f;
  bool sel = in && rank < a.k;
  float sum = a.renorm ? wave_sum(sel ? s : 0.f) : 1.f;
  // (scores that 32 bits hardly hold, too: all of them, or one beside others of which it is a share)
  if (__any(in && near) || sum < 0x1p-90f || (a.renorm && sum < 0.5f && __any(sel && s < 0x1p-126f && x > -INFINITY))) {
    if (a.softmax) base.total = total64<P>(sc, a.E, base.top);
    const double wide = in ? score64(a, base, x) : 0.0;
    const uint64_t best = !in ? 0ull : x == -INFINITY ? kOff : a.bias ? orderable64(wide + (double)a.bias[e]) : orderable64((double)x);
    rank = 0;
    for (int j = 0; j < n; ++j) {
      const uint64_t o = from_lane(best, j);
      const int oe = __builtin_amdgcn_readlane(e, j);
      rank += o > best || (o == best && oe < e);
    }
    sel = in && rank < a.k;
    const double all = a.renorm ? wave_sum64(sel ? wide : 0.0) : 1.0;
    s = all == 0.0 ? 0.f : (float)(wide / all);
    sum = 1.f;
  }
  if (sel) {
    a.idx[(size_t)t * a.k + rank] = e;
    a.gates[(size_t)t * a.k + rank] = a.scale * (s / sum);
  }
}

// The gradient. A row's entries are gathered in LDS, zero where nothing was selected, and stored side by side. Bound by the
// bytes of the rows that it writes; logits are read where one was selected, or with softmax and without
// renormalisation all of them.
template <int P>
__global__ __launch_bounds__(64 * kWaves) void scores_backward(ScoreArgs a, bool vec) {
  __shared__ __attribute__((aligned(16))) float rows[kWaves][64 * P];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  float* row = rows[wave];
  const int32_t* idx = a.idx + (size_t)t * a.k;
  const float* dg = a.d_gates + (size_t)t * a.k;
  const bool full = a.softmax && !a.renorm;
  // assignment `lane`, and its logit
  int e = lane < a.k ? idx[lane] : -1;
  if ((unsigned)e >= (unsigned)a.E) e = -1;
  const float d0 = e >= 0 ? a.scale * dg[lane] : 0.f, l0 = e >= 0 ? logit_at(a, t, e) : -INFINITY;
  float l[P];
  if (full) {
#pragma unroll
    for (int i = 0; i < P; ++i) l[i] = lane + 64 * i < a.E ? logit_at(a, t, lane + 64 * i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) row[lane + 64 * i] = 0.f;
  Base base{0.f, 1.0};
  if (a.softmax) {  // over the row, or with renorm over what was selected
    float top = -INFINITY;
    bool nan = false;  // (a maximum leaves it out)
    auto look = [&](float v) {
      top = fmaxf(top, v);
      nan |= v != v;
    };
    if (full) {
#pragma unroll
      for (int i = 0; i < P; ++i) look(l[i]);
    } else {
      look(l0);
      for (int j = 64 + lane; j < a.k; j += 64)
        if ((unsigned)idx[j] < (unsigned)a.E) look(logit_at(a, t, idx[j]));
    }
    top = wave_maxf(top);
    base.top = __any(nan) || top == INFINITY ? NAN : top;  // (such a row has no scores)
    if (full) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) v += base.top == -INFINITY ? 0.f : expf(l[i] - base.top);
      base.total = wave_sum(v);
    }
  }
  auto score = [&](float v) {
    if (!a.softmax) return 1.f / (1.f + expf(-v));
    return base.top == -INFINITY ? 0.f : expf(v - base.top) / (float)base.total;
  };
  const float s0 = e >= 0 ? score(l0) : 0.f;
  float S = s0, D = d0 * s0;  // sums of the selected scores, and of d times them
  bool under = l0 > -INFINITY && s0 < 0x1p-126f;
  for (int j = 64 + lane; j < a.k; j += 64)
    if ((unsigned)idx[j] < (unsigned)a.E) {
      const float v = logit_at(a, t, idx[j]), s = score(v);
      under |= v > -INFINITY && s < 0x1p-126f;
      S += s;
      D = fmaf(a.scale * dg[j], s, D);
    }
  S = wave_sum(S);
  D = wave_sum(D);
  // Sigmoids that 32 bits hardly hold, all or one beside a small sum: their ratios are those of exp(l - most) / (1 + exp(l)). (The
  // gates come of 64 bits there, in which a score is 0 from the limit here down. Softmax scores are 1 at most's place.)
  const bool tiny = a.renorm && (S < 0x1p-90f || (S < 0.5f && __any(under)));
  float most = l0;
  auto low = [&](float v) { return v <= -709.78271484375f ? 0.f : expf(v - most) / (1.f + expf(v)); };
  float part = s0;
  if (tiny) {
    for (int j = 64 + lane; j < a.k; j += 64)
      if ((unsigned)idx[j] < (unsigned)a.E) most = fmaxf(most, logit_at(a, t, idx[j]));
    most = wave_maxf(most);
    S = part = low(l0);
    D = d0 * part;
    for (int j = 64 + lane; j < a.k; j += 64)
      if ((unsigned)idx[j] < (unsigned)a.E) {
        const float s = low(logit_at(a, t, idx[j]));
        S += s;
        D = fmaf(a.scale * dg[j], s, D);
      }
    S = wave_sum(S);
    D = wave_sum(D);
  }
  const float mean = a.renorm ? (S == 0.f ? 0.f : D / S) : 0.f, inv = a.renorm ? (S == 0.f ? 0.f : 1.f / S) : 1.f;
  __builtin_amdgcn_wave_barrier();
  // An entry's value from the sum of its d: the first of an expert's assignments adds them up, in order. `part` over the sum is its
  // share of the gates (d over the sum by itself may pass the range); 1 - s of a sigmoid is exp(-v) s where s is near 1.
  auto entry = [&](float d, float part, float s, float v) {
    if (full) return d;
    const float g = d * (part * inv);
    return a.softmax ? g : g * (v < 0.f ? 1.f - s : expf(-v) * s);
  };
  if (a.k <= 64) {
    const float mine = d0 - mean;
    float sum = 0.f;
    bool first = e >= 0;
    for (int j = 0; j < a.k; ++j) {
      const int oe = __builtin_amdgcn_readlane(e, j);
      const float od = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), j));
      if (oe == e) {
        sum += od;
        first &= j >= lane;
      }
    }
    if (first) row[e] = entry(sum, part, s0, l0);
  } else {
    for (int j = 0; j < a.k; ++j) {
      const int o = idx[j];
      if ((unsigned)o < (unsigned)a.E && lane == 0) row[o] += a.scale * dg[j] - mean;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int c = lane; !full && c < a.E; c += 64)
      if (row[c] != 0.f) {
        const float v = logit_at(a, t, c), s = score(v);
        row[c] = entry(row[c], tiny ? low(v) : s, s, v);
      }
  }
  __builtin_amdgcn_wave_barrier();
  if (full) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 64 * i < a.E) row[lane + 64 * i] = score(l[i]) * (row[lane + 64 * i] - D);
    __builtin_amdgcn_wave_barrier();
  }
  const size_t at = (size_t)t * a.E;
#pragma unroll
  for (int i = 0; i < P; i += 4) {
    if (vec) {  // four neighbours a lane
      const int c = 4 * lane + 64 * i;
      if (c >= a.E) continue;
      const float4 v = *reinterpret_cast<const float4*>(row + c);
      if (a.bf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dlogits) + at + c) =
            make_uint2(f32_to_bf16_bits(v.x) | f32_to_bf16_bits(v.y) << 16, f32_to_bf16_bits(v.z) | f32_to_bf16_bits(v.w) << 16);
      else
        *reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + at + c) = v;
    } else {
#pragma unroll
      for (int z = 0; z < 4 && i + z < P; ++z) {
        const int c = lane + 64 * (i + z);
        if (c >= a.E) continue;
        if (a.bf16) static_cast<uint16_t*>(a.dlogits)[at + c] = (uint16_t)f32_to_bf16_bits(row[c]);
        else static_cast<float*>(a.dlogits)[at + c] = row[c];
      }
    }
  }
}

}  // namespace

#define BY_LANES(M) \
  const int per = (a.E + 63) / 64; \
  if (per <= 1) { M(1); } \
  else if (per <= 2) { M(2); } \
  else if (per <= 4) { M(4); } \
  else if (per <= 8) { M(8); } \
  else if (per <= 16) { M(16); } \
  else { M(32); }

hipError_t launch_scores(const ScoreArgs& a, hipStream_t s) {
  const dim3 g((a.T + kWaves - 1) / kWaves);
#define FORWARD(P) MOE_LAUNCH("scores", s, scores_forward<P>, g, dim3(64 * kWaves), 0, s, a)
  BY_LANES(FORWARD)
#undef FORWARD
  return hipGetLastError();
}

hipError_t launch_scores_backward(const ScoreArgs& a, hipStream_t s) {
  const dim3 g((a.T + kWaves - 1) / kWaves);
  const bool vec = a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.dlogits) & 15) == 0;
#define BACKWARD(P) MOE_LAUNCH("scores_backward", s, scores_backward<P>, g, dim3(64 * kWaves), 0, s, a, vec)
  BY_LANES(BACKWARD)
#undef BACKWARD
  return hipGetLastError();
}

}  // namespace moe
