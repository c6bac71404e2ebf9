// Host implementation of the 8-bit calls, the RMS norm and routing by scores of
// include/moe.h: argument checks and dispatch. Nothing here allocates.
#include <math.h>

#include "checks.h"
#include "f8.h"
#include "norm.h"

namespace {

constexpr int32_t kMaxDim = 1 << 19;
constexpr int32_t kMaxRows = moe::kMx4MaxRows;
constexpr long long kMaxLd = 1LL << 40;

typedef unsigned long long u64;

u64 row_bytes(int64_t rows, int32_t n) { return (u64)rows * moe::f8_blocks(n) * moe::kF8Block; }
u64 row_scale_bytes(int64_t rows, int32_t n) { return (u64)rows * moe::f8_blocks(n) * sizeof(float); }
u64 matrix_scale_bytes(int64_t mats, int32_t N, int32_t K) {
  return (u64)mats * moe::f8_blocks(N) * moe::f8_blocks(K) * sizeof(float);
}

// Checks that all products share: rows of n_in values come in, n_out values a row go out.
int check_product(const uint8_t* x, const float* xs, int64_t rows, const uint8_t* wc, const float* ws, int32_t N, int32_t K,
                  const void* y, int32_t out) {
  if (rows < 0 || N < 1 || K < 1 || !float_type(out)) return MOE_ERR_INVALID_ARG;
  if (N > kMaxDim || K > kMaxDim || rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !xs || !wc || !ws || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(wc, 16) || !aligned(xs, 4) || !aligned(ws, 4) || !aligned(y, size_of(out)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool overlaps_operands(const void* y, u64 n, const uint8_t* x, const float* xs, int64_t rows, int32_t n_in, const uint8_t* wc,
                       const float* ws, int64_t mats, int32_t N, int32_t K) {
  return overlaps(y, n, flat(wc, row_bytes(mats * N, K))) || overlaps(y, n, flat(ws, matrix_scale_bytes(mats, N, K))) ||
         overlaps(y, n, flat(x, row_bytes(rows, n_in))) || overlaps(y, n, flat(xs, row_scale_bytes(rows, n_in)));
}

int check_groups(int32_t T, int32_t k, int32_t E, int32_t has_shared, int32_t gather) {
  if (T < 0 || k < 1 || E < 1 || (has_shared != 0 && has_shared != 1) || (gather != 0 && gather != 1))
    return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_E + 1 - has_shared || k > kMaxRows || (k + (long long)has_shared) * T > kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Bytes of the counters (eight, 128 bytes apart) from which the gradient's workgroups may take tiles (which launches do: f8_tiles.hip),
// from this many rows on: 2,112 rows of [1024, 2048] 193 us taken, 198 dealt, unevenly loaded 52 and 48.
constexpr int32_t kCounterRows = 2048;
size_t counter_bytes(long long rows) { return rows >= kCounterRows ? 1024 : 0; }

moe::F8Args product(const uint8_t* x, const float* xs, int32_t A, const uint8_t* wc, const float* ws, int32_t N, int32_t K,
                    void* y, int32_t out, bool back) {
  moe::F8Args a{};
  a.x = x;
  a.xf = xs;
  a.A = A;
  a.T = A;
  a.k = 1;
  a.E_tot = 1;
  a.wc = wc;
  a.wf = ws;
  a.N = back ? K : N;
  a.K = back ? N : K;
  a.xb = moe::f8_blocks(a.K);
  a.wb = moe::f8_blocks(K);
  a.y = y;
  a.ydtype = out;
  a.back = back;
  a.exact = out != MOE_BF16;
  return a;
}

bool strided(int64_t ld, int32_t n) { return ld >= n; }

}  // namespace

extern "C" {

int moe_fp8_quantize(const void* x, int32_t xdtype, int64_t ld, int32_t mats, int32_t rows, int32_t K,
                     int32_t block_rows, uint8_t* codes, float* scales, void* stream) {
  if (mats < 0 || rows < 0 || K < 1 || ld < K || !float_type(xdtype) || (block_rows != 1 && block_rows != 128))
    return MOE_ERR_INVALID_ARG;
  if (K > kMaxDim || ld > kMaxLd || (long long)mats * rows > 0x7FFFFFFFLL) return MOE_ERR_UNSUPPORTED;
  if (mats == 0 || rows == 0) return MOE_OK;
  const long long of = block_rows == 1 ? (long long)mats * rows : (long long)mats * moe::f8_blocks(rows);
  // a workgroup a matrix block, and at most 2^32 threads a launch
  if (block_rows == 128 && of * moe::f8_blocks(K) >= 1 << 24) return MOE_ERR_UNSUPPORTED;
  if (!x || !codes || !scales || !aligned(x, size_of(xdtype)) || !aligned(codes, 16) || !aligned(scales, 4))
    return MOE_ERR_INVALID_ARG;
  const u64 cb = row_bytes((long long)mats * rows, K), sb = (u64)of * moe::f8_blocks(K) * sizeof(float);
  const Rows in = float_rows(x, xdtype, ld, (long long)mats * rows, K);
  if (overlaps(codes, cb, in) || overlaps(scales, sb, in) || overlaps(codes, cb, flat(scales, sb))) return MOE_ERR_INVALID_ARG;
  return status_of(moe::launch_f8_quantize(x, xdtype, ld, mats, rows, K, block_rows, codes, scales,
                                           static_cast<hipStream_t>(stream)));
}

int moe_fp8_dequantize(const uint8_t* codes, const float* scales, int32_t mats, int32_t rows, int32_t K,
                       int32_t block_rows, int32_t ydtype, void* y, void* stream) {
  if (mats < 0 || rows < 0 || K < 1 || !float_type(ydtype) || (block_rows != 1 && block_rows != 128))
    return MOE_ERR_INVALID_ARG;
  if (K > kMaxDim || (long long)mats * rows > 0x7FFFFFFFLL) return MOE_ERR_UNSUPPORTED;
  if (mats == 0 || rows == 0) return MOE_OK;
  if (!codes || !scales || !y || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(y, size_of(ydtype)))
    return MOE_ERR_INVALID_ARG;
  const long long of = block_rows == 1 ? (long long)mats * rows : (long long)mats * moe::f8_blocks(rows);
  const u64 out = (u64)mats * rows * K * size_of(ydtype);
  if (overlaps(y, out, flat(codes, row_bytes((long long)mats * rows, K))) ||
      overlaps(y, out, flat(scales, (u64)of * moe::f8_blocks(K) * sizeof(float))))
    return MOE_ERR_INVALID_ARG;
  return status_of(moe::launch_f8_dequantize(codes, scales, mats, rows, K, block_rows, ydtype, y,
                                             static_cast<hipStream_t>(stream)));
}

int moe_fp8_matmul(const uint8_t* x_codes, const float* x_scales, int32_t T, const uint8_t* w_codes,
                   const float* w_scales, int32_t N, int32_t K, void* y, int32_t ydtype, void* stream) {
  const int st = check_product(x_codes, x_scales, T, w_codes, w_scales, N, K, y, ydtype);
  if (st != MOE_OK || T == 0) return st;
  if (overlaps_operands(y, (u64)T * N * size_of(ydtype), x_codes, x_scales, T, K, w_codes, w_scales, 1, N, K))
    return MOE_ERR_INVALID_ARG;
  const moe::F8Args a = product(x_codes, x_scales, T, w_codes, w_scales, N, K, y, ydtype, false);
  return status_of(moe::launch_f8_product(a, static_cast<hipStream_t>(stream)));
}

int moe_fp8_matmul_backward(const uint8_t* dy_codes, const float* dy_scales, int32_t T, const uint8_t* w_codes,
                            const float* w_scales, int32_t N, int32_t K, void* dx, int32_t dxdtype, void* stream) {
  const int st = check_product(dy_codes, dy_scales, T, w_codes, w_scales, N, K, dx, dxdtype);
  if (st != MOE_OK || T == 0) return st;
  if (overlaps_operands(dx, (u64)T * K * size_of(dxdtype), dy_codes, dy_scales, T, N, w_codes, w_scales, 1, N, K))
    return MOE_ERR_INVALID_ARG;
  const moe::F8Args a = product(dy_codes, dy_scales, T, w_codes, w_scales, N, K, dx, dxdtype, true);
  return status_of(moe::launch_f8_product(a, static_cast<hipStream_t>(stream)));
}

int moe_fp8_experts_matmul(const uint8_t* x_codes, const float* x_scales, int32_t T, int32_t k, int32_t E,
                           int32_t has_shared, int32_t gather, const int32_t* offsets, const int32_t* perm,
                           const uint8_t* w_codes, const float* w_scales, int32_t N, int32_t K, void* y, int32_t ydtype,
                           void* stream) {
  int st = check_groups(T, k, E, has_shared, gather);
  if (st != MOE_OK) return st;
  const int32_t A = T * (k + has_shared), mats = E + has_shared;
  st = check_product(x_codes, x_scales, A, w_codes, w_scales, N, K, y, ydtype);
  if (st != MOE_OK || A == 0) return st;
  if (!offsets || (gather && !perm)) return MOE_ERR_INVALID_ARG;
  const u64 out = (u64)A * N * size_of(ydtype), ids = sizeof(int32_t) * (u64)A, ends = sizeof(int32_t) * (u64)(mats + 1);
  const int32_t rows = gather ? T : A;
  if (overlaps_operands(y, out, x_codes, x_scales, rows, K, w_codes, w_scales, mats, N, K) ||
      overlaps(y, out, flat(offsets, ends)) || (gather && overlaps(y, out, flat(perm, ids))))
    return MOE_ERR_INVALID_ARG;
  moe::F8Args a = product(x_codes, x_scales, A, w_codes, w_scales, N, K, y, ydtype, false);
  a.T = T;
  a.k = k;
  a.E_tot = mats;
  a.offsets = offsets;
  a.perm = gather ? perm : nullptr;
  return status_of(moe::launch_f8_product(a, static_cast<hipStream_t>(stream)));
}

size_t moe_fp8_experts_matmul_backward_workspace_size(int32_t T, int32_t k, int32_t has_shared, int32_t K,
                                                      int32_t gather) {
  if (K < 1 || check_groups(T, k, 1, has_shared, gather) != MOE_OK) return 0;
  const size_t A = (size_t)T * (k + has_shared);
  return counter_bytes(A) + (gather ? sizeof(float) * A * K : 0);
}

int moe_fp8_experts_matmul_backward(const uint8_t* dy_codes, const float* dy_scales, int32_t T, int32_t k, int32_t E,
                                    int32_t has_shared, int32_t gather, const int32_t* offsets, const int32_t* slot_of,
                                    const uint8_t* w_codes, const float* w_scales, int32_t N, int32_t K, void* dx,
                                    int32_t dxdtype, void* ws, size_t ws_bytes, void* stream) {
  int st = check_groups(T, k, E, has_shared, gather);
  if (st != MOE_OK) return st;
  const int32_t A = T * (k + has_shared), mats = E + has_shared;
  st = check_product(dy_codes, dy_scales, A, w_codes, w_scales, N, K, dx, dxdtype);
  if (st != MOE_OK || A == 0) return st;
  if (!offsets || (gather && !slot_of)) return MOE_ERR_INVALID_ARG;
  const size_t need = moe_fp8_experts_matmul_backward_workspace_size(T, k, has_shared, K, gather);
  if (need && (!ws || !aligned(ws, 16) || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  const u64 out = (u64)(gather ? T : A) * K * size_of(dxdtype), ids = sizeof(int32_t) * (u64)A,
            ends = sizeof(int32_t) * (u64)(mats + 1);
  if (overlaps_operands(dx, out, dy_codes, dy_scales, A, N, w_codes, w_scales, mats, N, K) ||
      overlaps(dx, out, flat(offsets, ends)) || (gather && overlaps(dx, out, flat(slot_of, ids))) ||
      (need && (overlaps(dx, out, flat(ws, need)) || overlaps(ws, need, flat(offsets, ends)) ||
                (gather && overlaps(ws, need, flat(slot_of, ids))) ||
                overlaps_operands(ws, need, dy_codes, dy_scales, A, N, w_codes, w_scales, mats, N, K))))
    return MOE_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  void* part = gather ? static_cast<char*>(ws) + counter_bytes(A) : nullptr;
  moe::F8Args a = product(dy_codes, dy_scales, A, w_codes, w_scales, N, K, gather ? part : dx, gather ? MOE_F32 : dxdtype, true);
  a.exact = dxdtype != MOE_BF16;
  a.counter = counter_bytes(A) ? static_cast<uint32_t*>(ws) : nullptr;
  a.E_tot = mats;
  a.offsets = offsets;
  hipError_t e = moe::launch_f8_product(a, s);
  if (e == hipSuccess && gather)
    e = moe::launch_mx4_sum_tokens(static_cast<const float*>(part), slot_of, offsets, mats, T, k, has_shared, A, K, dx,
                                   dxdtype, s);
  return status_of(e);
}

int moe_rms_norm(const void* x, int32_t dtype, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                 int32_t wdtype, float eps, int32_t T, int32_t H, void* total, void* y, uint8_t* codes, float* scales,
                 void* stream) {
  if (T < 0 || H < 1 || !float_type(dtype) || !float_type(wdtype) || !strided(ldx, H) || (residual && !strided(ldr, H)))
    return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || isinf(eps) || (codes != nullptr) != (scales != nullptr)) return MOE_ERR_INVALID_ARG;
  if (H > MOE_MAX_NORM_H || T > kMaxRows || ldx > kMaxLd || (residual && ldr > kMaxLd)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const unsigned size = size_of(dtype);
  if (!x || !weight || (!total && !y && !codes) || !aligned(x, size) || !aligned(residual, size) ||
      !aligned(weight, size_of(wdtype)) || !aligned(total, size) || !aligned(y, size) || !aligned(codes, 16) ||
      !aligned(scales, 4))
    return MOE_ERR_INVALID_ARG;
  const u64 n = (u64)T * H * size, cb = row_bytes(T, H), sb = row_scale_bytes(T, H);
  const Rows in[3] = {float_rows(x, dtype, ldx, T, H), float_rows(residual, dtype, ldr, T, H),
                      flat(weight, (u64)H * size_of(wdtype))};
  const Rows out[4] = {flat(total, n), flat(y, n), flat(codes, cb), flat(scales, sb)};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 3; ++i) {
      // a row of the sum in its operand's own place: whoever writes a value has read it
      const bool own = o == 0 && ((i == 0 && total == x && ldx == H) || (i == 1 && total == residual && ldr == H));
      if (!own && overlaps(out[o].p, out[o].bytes, in[i])) return MOE_ERR_INVALID_ARG;
    }
    for (int z = 0; z < o; ++z)
      if (overlaps(out[o].p, out[o].bytes, out[z])) return MOE_ERR_INVALID_ARG;
  }
  return status_of(moe::launch_norm(x, dtype, ldx, residual, ldr, weight, wdtype, eps, T, H, total, y, codes, scales,
                                    static_cast<hipStream_t>(stream)));
}

size_t moe_rms_norm_backward_workspace_size(int32_t T, int32_t H) {
  if (T < 1 || H < 1 || H > MOE_MAX_NORM_H || T > kMaxRows) return 0;
  return moe::norm_workspace_bytes(T, H);
}

int moe_rms_norm_backward(const void* dy, int64_t ldd, const void* h, int64_t ldh, int32_t dtype, const void* weight,
                          int32_t wdtype, const void* d_total, int64_t ldt, float eps, int32_t T, int32_t H, void* dh,
                          float* dweight, void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || H < 1 || !float_type(dtype) || !float_type(wdtype) || !strided(ldd, H) || !strided(ldh, H) ||
      (d_total && !strided(ldt, H)) || !(eps >= 0.f) || isinf(eps))
    return MOE_ERR_INVALID_ARG;
  if (H > MOE_MAX_NORM_H || T > kMaxRows || ldd > kMaxLd || ldh > kMaxLd || (d_total && ldt > kMaxLd))
    return MOE_ERR_UNSUPPORTED;
  if (!aligned(dweight, 4)) return MOE_ERR_INVALID_ARG;
  const unsigned size = size_of(dtype);
  if (T > 0) {
    if (!dy || !h || !weight || !dh || !aligned(dy, size) || !aligned(h, size) || !aligned(d_total, size) ||
        !aligned(dh, size) || !aligned(weight, size_of(wdtype)))
      return MOE_ERR_INVALID_ARG;
    const size_t need = dweight ? moe::norm_workspace_bytes(T, H) : 0;
    if (need && (!ws || !aligned(ws, 16) || ws_bytes < need)) return MOE_ERR_WORKSPACE;
    const Rows in[4] = {float_rows(dy, dtype, ldd, T, H), float_rows(h, dtype, ldh, T, H),
                        float_rows(d_total, dtype, ldt, T, H), flat(weight, (u64)H * size_of(wdtype))};
    const Rows out[3] = {flat(dh, (u64)T * H * size), flat(dweight, sizeof(float) * (u64)H), flat(need ? ws : nullptr, need)};
    for (int o = 0; o < 3; ++o) {
      for (int i = 0; i < 4; ++i)
        if (overlaps(out[o].p, out[o].bytes, in[i])) return MOE_ERR_INVALID_ARG;
      for (int z = 0; z < o; ++z)
        if (overlaps(out[o].p, out[o].bytes, out[z])) return MOE_ERR_INVALID_ARG;
    }
  } else if (!dweight) {
    return MOE_OK;
  }
  return status_of(moe::launch_norm_backward(dy, ldd, h, ldh, dtype, weight, wdtype, d_total, ldt, eps, T, H, dh, dweight,
                                             ws, static_cast<hipStream_t>(stream)));
}

int moe_route_scores(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E, const float* bias,
                     int32_t score, int32_t groups, int32_t keep, int32_t group_top, int32_t k, int32_t renorm,
                     float scale, int32_t* idx, float* gates, void* stream) {
  if (T < 0 || E < 1 || !strided(ld, E) || !float_type(dtype) || (score != MOE_SIGMOID && score != MOE_SOFTMAX) || groups < 1 ||
      keep < 1 || keep > groups || (group_top != 1 && group_top != 2) || k < 1 || E % groups || isnan(scale) || isinf(scale))
    return MOE_ERR_INVALID_ARG;
  if (k > (long long)keep * (E / groups)) return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_E || groups > 64 || T > kMaxRows || ld > kMaxLd) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !idx || !gates || !aligned(logits, size_of(dtype)) || !aligned(bias, 4) || !aligned(idx, 4) || !aligned(gates, 4))
    return MOE_ERR_INVALID_ARG;
  const u64 n = sizeof(int32_t) * (u64)T * k;
  const Rows in = float_rows(logits, dtype, ld, T, E), b = flat(bias, sizeof(float) * (u64)E);
  if (overlaps(idx, n, in) || overlaps(gates, n, in) || overlaps(idx, n, b) || overlaps(gates, n, b) ||
      overlaps(idx, n, flat(gates, n)))
    return MOE_ERR_INVALID_ARG;
  moe::ScoreArgs a{logits, ld, dtype == MOE_BF16, T, E, k, bias, score == MOE_SOFTMAX, groups, keep, group_top, renorm != 0,
                   scale, idx, gates, nullptr, nullptr};
  return status_of(moe::launch_scores(a, static_cast<hipStream_t>(stream)));
}

int moe_route_scores_backward(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E, int32_t k,
                              int32_t score, int32_t renorm, float scale, const int32_t* idx, const float* d_gates,
                              void* dlogits, void* stream) {
  if (T < 0 || E < 1 || !strided(ld, E) || !float_type(dtype) || (score != MOE_SIGMOID && score != MOE_SOFTMAX) || k < 1 ||
      isnan(scale) || isinf(scale))
    return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_E || k > MOE_MAX_E || T > kMaxRows || ld > kMaxLd) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !idx || !d_gates || !dlogits || !aligned(logits, size_of(dtype)) || !aligned(dlogits, size_of(dtype)) ||
      !aligned(idx, 4) || !aligned(d_gates, 4))
    return MOE_ERR_INVALID_ARG;
  const u64 n = sizeof(int32_t) * (u64)T * k, out = (u64)T * E * size_of(dtype);
  if (overlaps(dlogits, out, float_rows(logits, dtype, ld, T, E)) || overlaps(dlogits, out, flat(idx, n)) ||
      overlaps(dlogits, out, flat(d_gates, n)))
    return MOE_ERR_INVALID_ARG;
  moe::ScoreArgs a{logits, ld, dtype == MOE_BF16, T, E, k, nullptr, score == MOE_SOFTMAX, 1, 1, 1, renorm != 0, scale,
                   const_cast<int32_t*>(idx), nullptr, d_gates, dlogits};
  return status_of(moe::launch_scores_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
