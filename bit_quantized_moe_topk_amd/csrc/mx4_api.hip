// Host implementation of the microscaled 4-bit calls and the balance loss of
// include/moe.h: argument checks and dispatch. Nothing here allocates.
#include "../../include/moe.h"
#include "balance.h"
#include "mx4.h"

namespace {

inline int status_of(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool float_type(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
inline unsigned size_of(int32_t t) { return t == MOE_BF16 ? 2u : 4u; }

// Limits of the launches: rows and columns of a matrix, rows of a product.
constexpr int32_t kMaxDim = 1 << 19;
constexpr int32_t kMaxRows = moe::kMx4MaxRows;
// Assignments of a balance loss: row numbers and ids, and a launch's strides past them, fit 32 bits.
constexpr long long kMaxIds = 1LL << 30;

// Rows of `bytes` bytes, `step` bytes from one to the next, in memory.
struct Rows {
  const void* p;
  long long rows;
  unsigned long long bytes, step;
};
inline Rows flat(const void* p, unsigned long long bytes) { return {p, 1, bytes, bytes}; }
inline Rows float_rows(const void* p, int32_t type, int64_t ld, int64_t rows, int64_t n) {
  return {p, rows, (unsigned long long)n * size_of(type), (unsigned long long)ld * size_of(type)};
}

// Whether [y, y + n) holds a byte of one of those rows (128 bits: rows may reach past any address).
bool overlaps(const void* y, unsigned long long n, const Rows& r) {
  typedef unsigned __int128 wide;
  if (!y || !r.p || n == 0 || r.rows < 1 || r.bytes == 0) return false;
  const wide lo = reinterpret_cast<uintptr_t>(y), hi = lo + n, first = reinterpret_cast<uintptr_t>(r.p);
  if (hi <= first || lo >= first + (wide)(r.rows - 1) * r.step + r.bytes) return false;
  // the last row that starts at or before y, and the one after it
  const wide at = lo > first ? (lo - first) / r.step : 0;
  for (wide i = at; i < at + 2 && i < (wide)r.rows; ++i)
    if (lo < first + i * r.step + r.bytes && first + i * r.step < hi) return true;
  return false;
}

// The same of a product's results or workspace and its operands: rows x, codes wc and scales ws of `mats` matrices.
bool overlaps_operands(const void* y, unsigned long long n, const void* x, const uint8_t* xs, int32_t type, int64_t ld,
                       int64_t rows, int32_t n_in, const uint8_t* wc, const uint8_t* ws, int64_t mats, int32_t N, int32_t K) {
  const unsigned long long blocks = (unsigned long long)mats * N * moe::mx4_blocks(K);
  const unsigned long long xb = (unsigned long long)rows * moe::mx4_blocks(n_in);
  return overlaps(y, n, flat(wc, 16 * blocks)) || overlaps(y, n, flat(ws, blocks)) ||
         (type == MOE_MX4 ? overlaps(y, n, flat(x, 16 * xb)) || overlaps(y, n, flat(xs, xb))
                          : overlaps(y, n, float_rows(x, type, ld, rows, n_in)));
}

// Checks that all products share. dtype: of the rows that come in (n_in values
// each), out: of those that go out.
int check_product(const void* x, const uint8_t* xs, int32_t dtype, int64_t ld, int64_t rows, int32_t n_in,
                  const uint8_t* wc, const uint8_t* ws, int32_t N, int32_t K, const void* y, int32_t out) {
  if (rows < 0 || N < 1 || K < 1 || !float_type(out)) return MOE_ERR_INVALID_ARG;
  if (!float_type(dtype) && dtype != MOE_MX4) return MOE_ERR_INVALID_ARG;
  if ((dtype == MOE_MX4) != (xs != nullptr)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_MX4 && ld < n_in) return MOE_ERR_INVALID_ARG;
  if (N > kMaxDim || K > kMaxDim || rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (dtype != MOE_MX4 && ld > (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !wc || !ws || !y || !aligned(wc, 16)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, dtype == MOE_MX4 ? 16u : size_of(dtype)) || !aligned(y, size_of(out))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int check_groups(int32_t T, int32_t k, int32_t E, int32_t has_shared, int32_t gather) {
  if (T < 0 || k < 1 || E < 1 || (has_shared != 0 && has_shared != 1) || (gather != 0 && gather != 1))
    return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_E + 1 - has_shared || k > kMaxRows || (k + (long long)has_shared) * T > kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Bytes of the counters (eight, 128 bytes apart) from which workgroups take tiles, from this many rows on (fewer tiles than
// that many rows make are dealt in turn).
constexpr int32_t kCounterRows = 2048;
size_t counter_bytes(long long rows) { return rows >= kCounterRows ? 1024 : 0; }

moe::Mx4Args product(const void* x, const uint8_t* xs, int32_t dtype, int64_t ld, int32_t A, const uint8_t* wc,
                     const uint8_t* ws, int32_t N, int32_t K, void* y, int32_t out) {
  moe::Mx4Args a{};
  a.x = x;
  a.xs = xs;
  a.xdtype = dtype;
  a.ldx = ld;
  a.A = A;
  a.T = A;
  a.k = 1;
  a.E_tot = 1;
  a.wc = wc;
  a.ws = ws;
  a.N = N;
  a.K = K;
  a.y = y;
  a.ydtype = out;
  return a;
}

}  // namespace

extern "C" {

int moe_mx4_quantize(const void* x, int32_t xdtype, int64_t ld, int32_t rows, int32_t K, uint8_t* codes,
                     uint8_t* scales, void* stream) {
  if (rows < 0 || K < 1 || ld < K || !float_type(xdtype)) return MOE_ERR_INVALID_ARG;
  if (K > kMaxDim || ld > (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || !aligned(x, size_of(xdtype)) || !aligned(codes, 16)) return MOE_ERR_INVALID_ARG;
  const unsigned long long blocks = (unsigned long long)rows * moe::mx4_blocks(K);
  const Rows in = float_rows(x, xdtype, ld, rows, K);
  if (overlaps(codes, 16 * blocks, in) || overlaps(scales, blocks, in) || overlaps(codes, 16 * blocks, flat(scales, blocks)))
    return MOE_ERR_INVALID_ARG;
  return status_of(moe::launch_mx4_quantize(x, xdtype, ld, rows, K, codes, scales, static_cast<hipStream_t>(stream)));
}

int moe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t rows, int32_t K, int32_t ydtype,
                       void* y, void* stream) {
  if (rows < 0 || K < 1 || !float_type(ydtype)) return MOE_ERR_INVALID_ARG;
  if (K > kMaxDim) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !y || !aligned(codes, 16) || !aligned(y, size_of(ydtype))) return MOE_ERR_INVALID_ARG;
  const unsigned long long blocks = (unsigned long long)rows * moe::mx4_blocks(K);
  const unsigned long long out = (unsigned long long)rows * K * size_of(ydtype);
  if (overlaps(y, out, flat(codes, 16 * blocks)) || overlaps(y, out, flat(scales, blocks))) return MOE_ERR_INVALID_ARG;
  return status_of(moe::launch_mx4_dequantize(codes, scales, rows, K, ydtype, y, static_cast<hipStream_t>(stream)));
}

int moe_mx4_matmul(const void* x, const uint8_t* x_scales, int32_t xdtype, int64_t ldx, int32_t T,
                   const uint8_t* w_codes, const uint8_t* w_scales, int32_t N, int32_t K, void* y, int32_t ydtype,
                   void* stream) {
  const int st = check_product(x, x_scales, xdtype, ldx, T, K, w_codes, w_scales, N, K, y, ydtype);
  if (st != MOE_OK || T == 0) return st;
  if (overlaps_operands(y, (unsigned long long)T * N * size_of(ydtype), x, x_scales, xdtype, ldx, T, K, w_codes, w_scales,
                        1, N, K))
    return MOE_ERR_INVALID_ARG;
  const moe::Mx4Args a = product(x, x_scales, xdtype, ldx, T, w_codes, w_scales, N, K, y, ydtype);
  return status_of(moe::launch_mx4_forward(a, static_cast<hipStream_t>(stream)));
}

int moe_mx4_matmul_backward(const void* dy, int32_t dtype, int64_t ldd, int32_t T, const uint8_t* w_codes,
                            const uint8_t* w_scales, int32_t N, int32_t K, void* dx, int32_t dxdtype, void* stream) {
  if (!float_type(dtype)) return MOE_ERR_INVALID_ARG;
  const int st = check_product(dy, nullptr, dtype, ldd, T, N, w_codes, w_scales, N, K, dx, dxdtype);
  if (st != MOE_OK || T == 0) return st;
  if (overlaps_operands(dx, (unsigned long long)T * K * size_of(dxdtype), dy, nullptr, dtype, ldd, T, N, w_codes, w_scales,
                        1, N, K))
    return MOE_ERR_INVALID_ARG;
  const moe::Mx4Args a = product(dy, nullptr, dtype, ldd, T, w_codes, w_scales, N, K, dx, dxdtype);
  return status_of(moe::launch_mx4_gradient(a, static_cast<hipStream_t>(stream)));
}

size_t moe_mx4_experts_matmul_workspace_size(int32_t T, int32_t k, int32_t has_shared) {
  if (check_groups(T, k, 1, has_shared, 0) != MOE_OK) return 0;
  return counter_bytes((long long)T * (k + has_shared));
}

int moe_mx4_experts_matmul(const void* x, const uint8_t* x_scales, int32_t xdtype, int64_t ldx, int32_t T, int32_t k,
                           int32_t E, int32_t has_shared, int32_t gather, const int32_t* offsets, const int32_t* perm,
                           const uint8_t* w_codes, const uint8_t* w_scales, int32_t N, int32_t K, void* y,
                           int32_t ydtype, void* ws, size_t ws_bytes, void* stream) {
  int st = check_groups(T, k, E, has_shared, gather);
  if (st != MOE_OK) return st;
  const int32_t A = T * (k + has_shared);
  st = check_product(x, x_scales, xdtype, ldx, A, K, w_codes, w_scales, N, K, y, ydtype);
  if (st != MOE_OK || A == 0) return st;
  if (!offsets || (gather && !perm)) return MOE_ERR_INVALID_ARG;
  const size_t need = counter_bytes(A);
  if (need && (!ws || !aligned(ws, 16) || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  const unsigned long long out = (unsigned long long)A * N * size_of(ydtype);
  const int32_t rows = gather ? T : A;
  if (overlaps_operands(y, out, x, x_scales, xdtype, ldx, rows, K, w_codes, w_scales, E + has_shared, N, K) ||
      (need && (overlaps(y, out, flat(ws, need)) ||
                overlaps_operands(ws, need, x, x_scales, xdtype, ldx, rows, K, w_codes, w_scales, E + has_shared, N, K))))
    return MOE_ERR_INVALID_ARG;
  moe::Mx4Args a = product(x, x_scales, xdtype, ldx, A, w_codes, w_scales, N, K, y, ydtype);
  a.T = T;
  a.k = k;
  a.E_tot = E + has_shared;
  a.offsets = offsets;
  a.perm = gather ? perm : nullptr;
  a.counter = need ? static_cast<uint32_t*>(ws) : nullptr;
  return status_of(moe::launch_mx4_forward(a, static_cast<hipStream_t>(stream)));
}

size_t moe_mx4_experts_matmul_backward_workspace_size(int32_t T, int32_t k, int32_t has_shared, int32_t K,
                                                      int32_t gather) {
  if (K < 1 || check_groups(T, k, 1, has_shared, gather) != MOE_OK) return 0;
  const size_t A = (size_t)T * (k + has_shared);
  return counter_bytes(A) + (gather ? sizeof(float) * A * K : 0);
}

int moe_mx4_experts_matmul_backward(const void* dy, int32_t dtype, int64_t ldd, int32_t T, int32_t k, int32_t E,
                                    int32_t has_shared, int32_t gather, const int32_t* offsets,
                                    const int32_t* slot_of, const uint8_t* w_codes, const uint8_t* w_scales, int32_t N,
                                    int32_t K, void* dx, int32_t dxdtype, void* ws, size_t ws_bytes, void* stream) {
  if (!float_type(dtype)) return MOE_ERR_INVALID_ARG;
  int st = check_groups(T, k, E, has_shared, gather);
  if (st != MOE_OK) return st;
  const int32_t A = T * (k + has_shared);
  st = check_product(dy, nullptr, dtype, ldd, A, N, w_codes, w_scales, N, K, dx, dxdtype);
  if (st != MOE_OK || A == 0) return st;
  if (!offsets || (gather && !slot_of)) return MOE_ERR_INVALID_ARG;
  const size_t need = moe_mx4_experts_matmul_backward_workspace_size(T, k, has_shared, K, gather);
  if (need && (!ws || !aligned(ws, 16) || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  const unsigned long long out = (unsigned long long)(gather ? T : A) * K * size_of(dxdtype);
  if (overlaps_operands(dx, out, dy, nullptr, dtype, ldd, A, N, w_codes, w_scales, E + has_shared, N, K) ||
      (need && (overlaps(dx, out, flat(ws, need)) ||
                overlaps_operands(ws, need, dy, nullptr, dtype, ldd, A, N, w_codes, w_scales, E + has_shared, N, K))))
    return MOE_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  void* part = gather ? static_cast<char*>(ws) + counter_bytes(A) : nullptr;
  moe::Mx4Args a = product(dy, nullptr, dtype, ldd, A, w_codes, w_scales, N, K, gather ? part : dx,
                           gather ? MOE_F32 : dxdtype);
  a.counter = counter_bytes(A) ? static_cast<uint32_t*>(ws) : nullptr;
  a.E_tot = E + has_shared;
  a.offsets = offsets;
  hipError_t e = moe::launch_mx4_gradient(a, s);
  if (e == hipSuccess && gather)
    e = moe::launch_mx4_sum_tokens(static_cast<const float*>(part), slot_of, offsets, a.E_tot, T, k, has_shared, A, K,
                                   dx, dxdtype, s);
  return status_of(e);
}

size_t moe_balance_loss_workspace_size(int32_t T, int32_t k, int32_t E) {
  if (T < 0 || k < 1 || E < 1 || E > MOE_MAX_E || (long long)T * k > kMaxIds) return 0;
  return moe::balance_workspace_bytes(T, k, E);
}

int moe_balance_loss(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E, int32_t k,
                     const int32_t* idx, const uint8_t* mask, float* losses, int32_t* counts, int32_t* kept, void* ws,
                     size_t ws_bytes, void* stream) {
  if (T < 0 || E < 1 || k < 1 || ld < E || !float_type(dtype)) return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_E || (long long)T * k > kMaxIds || ld > (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  if (!losses || !counts || !kept || !aligned(losses, 4) || !aligned(counts, 4) || !aligned(kept, 4))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !idx || !aligned(logits, size_of(dtype)) || !aligned(idx, 4))) return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16) || ws_bytes < moe::balance_workspace_bytes(T, k, E)) return MOE_ERR_WORKSPACE;
  return status_of(moe::launch_balance(logits, dtype, ld, T, E, k, idx, mask, losses, counts, kept, ws,
                                       static_cast<hipStream_t>(stream)));
}

int moe_balance_loss_backward(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E, int32_t k,
                              const uint8_t* mask, const int32_t* counts, const int32_t* kept, const float* d_losses,
                              void* dlogits, void* stream) {
  if (T < 0 || E < 1 || k < 1 || ld < E || !float_type(dtype)) return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_E || (long long)T * k > kMaxIds || ld > (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !counts || !kept || !d_losses || !dlogits || !aligned(logits, size_of(dtype)) ||
      !aligned(dlogits, size_of(dtype)) || !aligned(counts, 4) || !aligned(kept, 4) || !aligned(d_losses, 4))
    return MOE_ERR_INVALID_ARG;
  // in the logits' own place every row is read by the wave that then writes it
  if (!(dlogits == logits && ld == E) &&
      overlaps(dlogits, (unsigned long long)T * E * size_of(dtype), float_rows(logits, dtype, ld, T, E)))
    return MOE_ERR_INVALID_ARG;
  return status_of(moe::launch_balance_gradient(logits, dtype, ld, T, E, k, mask, counts, kept, d_losses, dlogits,
                                                static_cast<hipStream_t>(stream)));
}

}  // extern "C"
