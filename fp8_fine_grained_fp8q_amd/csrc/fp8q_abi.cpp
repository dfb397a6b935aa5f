// C ABI of libfp8q (see include/fp8q.h): argument checks, then the call's kernel launches.
// Every check runs before the first HIP call, so a bad call never touches the device.
#include "fp8q.h"

#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdlib.h>

#include <mutex>

#include "fp8q_launch.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;
constexpr int64_t kMaxElems = int64_t(1) << 62;
constexpr int64_t kMaxGemmK = int64_t(1) << 22;

bool misaligned(const void *p, uintptr_t a = 16) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

bool bad_dim(int64_t v) { return v < 0 || v >= kMaxDim; }

bool too_many(int64_t a, int64_t b) { return a != 0 && b > kMaxElems / a; }

fp8q_status device_ok() {
  int dev = 0;
  return hipGetDevice(&dev) == hipSuccess ? FP8Q_OK : FP8Q_ERR_DEVICE;
}

fp8q_status launched(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_ERR_LAUNCH; }

hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }

// FP8Q_DEBUG set to anything but "" or "0" turns on the synchronizing argument checks.
bool debug_checks() {
  const char *v = getenv("FP8Q_DEBUG");
  return v != nullptr && v[0] != '\0' && !(v[0] == '0' && v[1] == '\0');
}

bool bad_dtype(int32_t d) { return d != FP8Q_OUT_BF16 && d != FP8Q_OUT_F32; }

// The kernels take their numbers in FP32: a finite one that stays finite there, and nonzero if it is.
bool f32_number(double v) { return fabs(v) <= FLT_MAX && (v == 0 || static_cast<float>(v) != 0.0f); }
bool f32_beta(double v) { return v >= 0 && static_cast<float>(v) < 1.0f; }

// Shared checks of the token maps [T][k] and of rows of `width` columns.
bool bad_rows(int64_t T, int64_t k, int64_t capacity, int64_t width) {
  return bad_dim(T) || k < 1 || k > 64 || bad_dim(width) || width % 8 != 0 || bad_dim(capacity) || too_many(T, k) ||
         T * k >= kMaxDim || too_many(capacity, width) || too_many(T, width);
}

// Shared checks of the two GEMM entry points (everything except the grouped extras).
fp8q_status check_gemm(const uint8_t *xq, const float *sa, const uint8_t *wq, const float *sb,
                       int64_t M, int64_t N, int64_t K, void *c, int32_t out_dtype) {
  if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return FP8Q_ERR_SHAPE;
  if (K < 128 || K % 128 != 0 || N % 128 != 0) return FP8Q_ERR_SHAPE;
  // The kernels address a stage of up to 512 operand rows with 32-bit buffer offsets
  // (row * K + byte), so K is limited to 2^22.
  if (K > kMaxGemmK) return FP8Q_ERR_SHAPE;
  if (too_many(M, K) || too_many(N, K) || too_many(M, N)) return FP8Q_ERR_SHAPE;
  if (M == 0 || N == 0) return 1;  // nothing to do (positive: caller returns FP8Q_OK)
  if (!xq || !sa || !wq || !sb || !c) return FP8Q_ERR_NULL;
  if (misaligned(xq) || misaligned(sa) || misaligned(wq) || misaligned(sb) || misaligned(c))
    return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

}  // namespace

extern "C" {

fp8q_status fp8q_quantize_act_1x128(const uint16_t *x_bf16, int64_t M, int64_t K, uint8_t *xq,
                                    float *sa, void *stream) {
  if (bad_dim(M) || bad_dim(K) || K % 128 != 0 || too_many(M, K)) return FP8Q_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8Q_OK;
  if (!x_bf16 || !xq || !sa) return FP8Q_ERR_NULL;
  if (misaligned(x_bf16) || misaligned(xq) || misaligned(sa)) return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_quant_act(x_bf16, M, K, xq, sa, as_stream(stream)));
}

fp8q_status fp8q_quantize_w_128x128(const uint16_t *w_bf16, int64_t G, int64_t N, int64_t K,
                                    uint8_t *wq, float *sb, void *stream) {
  if (G < 1 || bad_dim(G) || bad_dim(N) || bad_dim(K)) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (too_many(G, N) || too_many(G * N, K)) return FP8Q_ERR_SHAPE;
  if (N == 0 || K == 0) return FP8Q_OK;
  if (!w_bf16 || !wq || !sb) return FP8Q_ERR_NULL;
  if (misaligned(w_bf16) || misaligned(wq) || misaligned(sb)) return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_quant_w(w_bf16, G, N, K, wq, sb, nullptr, nullptr, as_stream(stream)));
}

fp8q_status fp8q_gemm_blockscaled(const uint8_t *xq, const float *sa, const uint8_t *wq,
                                  const float *sb, int64_t M, int64_t N, int64_t K, void *c,
                                  int32_t out_dtype, void *stream) {
  const fp8q_status st = check_gemm(xq, sa, wq, sb, M, N, K, c, out_dtype);
  if (st != FP8Q_OK) return st > 0 ? FP8Q_OK : st;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_gemm(xq, sa, wq, sb, M, N, K, c, out_dtype == FP8Q_OUT_F32,
                                    as_stream(stream)));
}

fp8q_status fp8q_grouped_gemm_blockscaled(const uint8_t *xq, const float *sa, const uint8_t *wq,
                                          const float *sb, const int32_t *offsets, int64_t G,
                                          int64_t M_tot, int64_t N, int64_t K, void *c,
                                          int32_t out_dtype, void *stream) {
  if (G < 1 || bad_dim(G)) return FP8Q_ERR_SHAPE;
  const fp8q_status st = check_gemm(xq, sa, wq, sb, M_tot, N, K, c, out_dtype);
  if (st < 0) return st;
  if (too_many(G, N) || too_many(G * N, K)) return FP8Q_ERR_SHAPE;
  if (st > 0) return FP8Q_OK;
  if (!offsets) return FP8Q_ERR_NULL;
  if (misaligned(offsets, 4)) return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  if (debug_checks()) {
    // One device flag serves the check: checks from several threads run one at a time.
    static std::mutex check_mutex;
    std::lock_guard<std::mutex> lock(check_mutex);
    bool bad = false;
    if (fp8q::check_grouped_offsets(offsets, G, M_tot, as_stream(stream), &bad) != hipSuccess)
      return FP8Q_ERR_LAUNCH;
    if (bad) return FP8Q_ERR_OFFSETS;
  }
  return launched(fp8q::launch_grouped_gemm(xq, sa, wq, sb, offsets, G, M_tot, N, K, c,
                                            out_dtype == FP8Q_OUT_F32, as_stream(stream)));
}

fp8q_status fp8q_quantize_act_w(const uint16_t *x_bf16, int64_t M, const uint16_t *w_bf16, int64_t G, int64_t N,
                                int64_t K, uint8_t *xq, float *sa, uint8_t *wq, float *sb, void *stream) {
  if (bad_dim(M) || bad_dim(K) || K % 128 != 0 || too_many(M, K)) return FP8Q_ERR_SHAPE;
  if (G < 1 || bad_dim(G) || bad_dim(N) || N % 128 != 0) return FP8Q_ERR_SHAPE;
  if (too_many(G, N) || too_many(G * N, K)) return FP8Q_ERR_SHAPE;
  const bool act = M > 0 && K > 0, wts = N > 0 && K > 0;
  if (!act && !wts) return FP8Q_OK;
  if (act && (!x_bf16 || !xq || !sa)) return FP8Q_ERR_NULL;
  if (wts && (!w_bf16 || !wq || !sb)) return FP8Q_ERR_NULL;
  if (act && (misaligned(x_bf16) || misaligned(xq) || misaligned(sa))) return FP8Q_ERR_ALIGN;
  if (wts && (misaligned(w_bf16) || misaligned(wq) || misaligned(sb))) return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_quant_act_w(x_bf16, act ? M : 0, xq, sa, w_bf16, G, wts ? N : 0, wq, sb, K,
                                           as_stream(stream)));
}

fp8q_status fp8q_quantize_w_128x128_t(const uint16_t *w_bf16, int64_t G, int64_t N, int64_t K,
                                      uint8_t *wq, float *sb, uint8_t *wqt, float *sbt, void *stream) {
  if (G < 1 || bad_dim(G) || bad_dim(N) || bad_dim(K)) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (too_many(G, N) || too_many(G * N, K)) return FP8Q_ERR_SHAPE;
  if (N == 0 || K == 0) return FP8Q_OK;
  if (!w_bf16 || !wq || !sb || !wqt || !sbt) return FP8Q_ERR_NULL;
  if (misaligned(w_bf16) || misaligned(wq) || misaligned(sb) || misaligned(wqt) || misaligned(sbt))
    return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_quant_w(w_bf16, G, N, K, wq, sb, wqt, sbt, as_stream(stream)));
}

fp8q_status fp8q_quantize_act_dual(const uint16_t *x_bf16, int64_t M, int64_t K, uint8_t *xq,
                                   float *sa, uint8_t *xqt, float *sat, void *stream) {
  if (bad_dim(M) || bad_dim(K) || M % 128 != 0 || K % 128 != 0 || too_many(M, K)) return FP8Q_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8Q_OK;
  if (!x_bf16 || !xq || !sa || !xqt || !sat) return FP8Q_ERR_NULL;
  if (misaligned(x_bf16) || misaligned(xq) || misaligned(sa) || misaligned(xqt) || misaligned(sat))
    return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_quant_act_dual(x_bf16, M, K, xq, sa, xqt, sat, as_stream(stream)));
}

fp8q_status fp8q_gemm_rowscaled(const uint8_t *aq, const float *sa, const uint8_t *bq, const float *sb,
                                int64_t P, int64_t Q, int64_t Kc, void *c, int32_t out_dtype,
                                void *stream) {
  const fp8q_status st = check_gemm(aq, sa, bq, sb, P, Q, Kc, c, out_dtype);
  if (st < 0) return st;
  if ((Kc / 128) * Q >= (int64_t(1) << 29)) return FP8Q_ERR_SHAPE;  // scale offsets fit 31 bits
  if (st > 0) return FP8Q_OK;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_gemm_rowscaled(aq, sa, bq, sb, P, Q, Kc, c, out_dtype == FP8Q_OUT_F32,
                                              as_stream(stream)));
}

fp8q_status fp8q_swiglu_quantize_act_1x128(const uint16_t *gu_bf16, int64_t M, int64_t I, uint8_t *xq,
                                           float *sa, void *stream) {
  if (bad_dim(M) || bad_dim(I) || I % 128 != 0 || too_many(M, 2 * I)) return FP8Q_ERR_SHAPE;
  if (M == 0 || I == 0) return FP8Q_OK;
  if (!gu_bf16 || !xq || !sa) return FP8Q_ERR_NULL;
  if (misaligned(gu_bf16) || misaligned(xq) || misaligned(sa)) return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_swiglu_quant_act(gu_bf16, M, I, xq, sa, as_stream(stream)));
}

fp8q_status fp8q_quantize_per_tensor(const uint16_t *x_bf16, int64_t n, const float *scale_in, uint8_t *q,
                                     uint32_t *stats, void *stream) {
  if (n < 0 || n % 8 != 0 || n >= kMaxElems) return FP8Q_ERR_SHAPE;
  if (!stats) return FP8Q_ERR_NULL;
  if (n > 0 && (!x_bf16 || !q)) return FP8Q_ERR_NULL;
  if (misaligned(x_bf16) || misaligned(q) || misaligned(stats, 4) || misaligned(scale_in, 4))
    return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_quant_per_tensor(x_bf16, n, scale_in, q, stats, as_stream(stream)));
}

fp8q_status fp8q_moe_dispatch(const int32_t *topk_ids, int64_t T, int64_t k, int64_t e_begin, int64_t E,
                              const uint8_t *xq, const float *sa, int64_t K, int64_t capacity, uint8_t *xq_sorted,
                              float *sa_sorted, int32_t *offsets, int32_t *token_row, int32_t *row_token,
                              void *stream) {
  if (bad_dim(T) || k < 1 || k > 64 || bad_dim(K) || K % 128 != 0 || E < 1 || E > 1024 || e_begin < 0 ||
      bad_dim(e_begin) || bad_dim(capacity))
    return FP8Q_ERR_SHAPE;
  if (too_many(T, k) || T * k >= kMaxDim || too_many(capacity, K) || too_many(T, K))
    return FP8Q_ERR_SHAPE;
  if (!offsets || (T > 0 && (!topk_ids || !token_row || !xq || !sa)) ||
      (capacity > 0 && (!xq_sorted || !sa_sorted || !row_token)))
    return FP8Q_ERR_NULL;
  if (misaligned(topk_ids, 4) || misaligned(offsets, 4) || misaligned(token_row, 4) || misaligned(row_token, 4) ||
      misaligned(xq) || misaligned(sa) || misaligned(xq_sorted) || misaligned(sa_sorted))
    return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_moe_dispatch(topk_ids, T, k, e_begin, E, xq, sa, K, capacity, xq_sorted, sa_sorted,
                                            offsets, token_row, row_token, as_stream(stream)));
}

fp8q_status fp8q_moe_combine(const void *expert_out, int32_t in_dtype, int64_t capacity, int64_t N,
                             const int32_t *token_row, const float *topk_weights, int64_t T, int64_t k, void *y,
                             int32_t out_dtype, void *stream) {
  if ((in_dtype != FP8Q_OUT_BF16 && in_dtype != FP8Q_OUT_F32) || (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32))
    return FP8Q_ERR_DTYPE;
  if (bad_dim(T) || k < 1 || k > 64 || bad_dim(N) || N % 8 != 0 || bad_dim(capacity) || too_many(T, k) ||
      too_many(capacity, N) || too_many(T, N))
    return FP8Q_ERR_SHAPE;
  if (T == 0 || N == 0) return FP8Q_OK;
  if (!token_row || !topk_weights || !y || (capacity > 0 && !expert_out)) return FP8Q_ERR_NULL;
  if (misaligned(token_row, 4) || misaligned(topk_weights, 4) || misaligned(y) || misaligned(expert_out))
    return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_moe_combine(expert_out, in_dtype == FP8Q_OUT_F32, capacity, N, token_row,
                                           topk_weights, T, k, y, out_dtype == FP8Q_OUT_F32, as_stream(stream)));
}

fp8q_status fp8q_moe_sort(const int32_t *topk_ids, int64_t T, int64_t k, int64_t e_begin, int64_t E, const void *x,
                          int32_t dtype, int64_t H, int64_t capacity, void *xs, int32_t *offsets, int32_t *token_row,
                          int32_t *row_token, void *stream) {
  if (bad_dtype(dtype)) return FP8Q_ERR_DTYPE;
  if (bad_rows(T, k, capacity, H) || E < 1 || E > 1024 || e_begin < 0 || bad_dim(e_begin)) return FP8Q_ERR_SHAPE;
  if (!fp8q::grid_fits(fp8q::moe_sort_groups(T, k, dtype == FP8Q_OUT_F32, H), 256)) return FP8Q_ERR_SHAPE;
  if (!offsets || (T > 0 && (!topk_ids || !token_row)) || (T > 0 && H > 0 && !x) ||
      (capacity > 0 && ((H > 0 && !xs) || !row_token)))
    return FP8Q_ERR_NULL;
  if (misaligned(topk_ids, 4) || misaligned(offsets, 4) || misaligned(token_row, 4) || misaligned(row_token, 4) ||
      misaligned(x) || misaligned(xs))
    return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_moe_sort(topk_ids, T, k, e_begin, E, x, dtype == FP8Q_OUT_F32, H, capacity, xs, offsets,
                                        token_row, row_token, as_stream(stream)));
}

fp8q_status fp8q_moe_sort_backward(const void *dxs, int32_t in_dtype, int64_t capacity, int64_t H,
                                   const int32_t *token_row, int64_t T, int64_t k, void *dx, int32_t out_dtype,
                                   void *stream) {
  if (bad_dtype(in_dtype) || bad_dtype(out_dtype)) return FP8Q_ERR_DTYPE;
  if (bad_rows(T, k, capacity, H)) return FP8Q_ERR_SHAPE;
  if (!fp8q::grid_fits(T * ((H + 2047) / 2048), 256)) return FP8Q_ERR_SHAPE;  // 2048 columns of a token each
  if (T == 0 || H == 0) return FP8Q_OK;
  if (!token_row || !dx || (capacity > 0 && !dxs)) return FP8Q_ERR_NULL;
  if (misaligned(token_row, 4) || misaligned(dx) || misaligned(dxs)) return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_moe_sort_backward(dxs, in_dtype == FP8Q_OUT_F32, capacity, H, token_row, T, k, dx,
                                                 out_dtype == FP8Q_OUT_F32, as_stream(stream)));
}

fp8q_status fp8q_moe_combine_backward(const void *dy, int32_t dy_dtype, const void *expert_out, int32_t dtype,
                                      int64_t capacity, int64_t N, const int32_t *token_row,
                                      const float *topk_weights, int64_t T, int64_t k, void *dout, float *dw,
                                      void *stream) {
  if (bad_dtype(dy_dtype) || bad_dtype(dtype)) return FP8Q_ERR_DTYPE;
  if (bad_rows(T, k, capacity, N)) return FP8Q_ERR_SHAPE;
  if (!fp8q::grid_fits((T * k + 3) / 4, 256)) return FP8Q_ERR_SHAPE;  // a wave per slot
  if (T == 0) return FP8Q_OK;
  if (!token_row || !topk_weights || !dw || (N > 0 && (!dy || (capacity > 0 && (!expert_out || !dout)))))
    return FP8Q_ERR_NULL;
  if (misaligned(token_row, 4) || misaligned(topk_weights, 4) || misaligned(dw, 4) || misaligned(dy) ||
      misaligned(expert_out) || misaligned(dout))
    return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_moe_combine_backward(dy, dy_dtype == FP8Q_OUT_F32, expert_out, dtype == FP8Q_OUT_F32,
                                                    capacity, N, token_row, topk_weights, T, k, dout, dw,
                                                    as_stream(stream)));
}

fp8q_status fp8q_swiglu_backward(const uint16_t *gu_bf16, const void *dh, int32_t dh_dtype, int64_t M, int64_t I,
                                 uint16_t *dgu_bf16, uint16_t *h_bf16, void *stream) {
  if (bad_dtype(dh_dtype)) return FP8Q_ERR_DTYPE;
  if (bad_dim(M) || bad_dim(I) || I % 8 != 0 || too_many(M, 2 * I)) return FP8Q_ERR_SHAPE;
  if (!fp8q::grid_fits((M * (I / 8) + 255) / 256, 256)) return FP8Q_ERR_SHAPE;  // eight elements of h per thread
  if (M == 0 || I == 0) return FP8Q_OK;
  if (!gu_bf16 || !dh || !dgu_bf16) return FP8Q_ERR_NULL;
  if (misaligned(gu_bf16) || misaligned(dh) || misaligned(dgu_bf16) || misaligned(h_bf16)) return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_swiglu_backward(gu_bf16, dh, dh_dtype == FP8Q_OUT_F32, M, I, dgu_bf16, h_bf16,
                                               as_stream(stream)));
}

fp8q_status fp8q_quantize_act_grouped(const uint16_t *x_bf16, const int32_t *offsets, int64_t G, int64_t M_tot,
                                      int64_t K, uint8_t *xq, float *sa, uint8_t *xqt, float *sat, void *stream) {
  if (G < 1 || bad_dim(G) || bad_dim(M_tot) || bad_dim(K) || K % 128 != 0 || too_many(M_tot, K))
    return FP8Q_ERR_SHAPE;
  // 128 channels of a tile per workgroup, or 64 without the rows' codes
  if (!fp8q::grid_fits((M_tot / 128 + G) * (K / (xq ? 128 : 64)), 256)) return FP8Q_ERR_SHAPE;
  if (M_tot == 0 || K == 0) return FP8Q_OK;
  if (!x_bf16 || !offsets || !xqt || !sat || !xq != !sa) return FP8Q_ERR_NULL;
  if (misaligned(x_bf16) || misaligned(offsets, 4) || misaligned(xq) || misaligned(sa) || misaligned(xqt) ||
      misaligned(sat))
    return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_quant_act_grouped(x_bf16, offsets, G, M_tot, K, xq, sa, xqt, sat,
                                                 as_stream(stream)));
}

fp8q_status fp8q_grouped_gemm_rowscaled(const uint8_t *aq, const float *sa, const uint8_t *bq, const float *sb,
                                        const int32_t *offsets, int64_t G, int64_t M_tot, int64_t P, int64_t Q,
                                        void *c, int32_t out_dtype, void *stream) {
  if (bad_dtype(out_dtype)) return FP8Q_ERR_DTYPE;
  if (G < 1 || bad_dim(G) || bad_dim(M_tot) || bad_dim(P) || bad_dim(Q) || P % 128 != 0 || Q % 128 != 0)
    return FP8Q_ERR_SHAPE;
  if (P > kMaxGemmK || Q > kMaxGemmK) return FP8Q_ERR_SHAPE;  // 32-bit offsets within a tile's rows
  if (too_many(G, P) || too_many(G * P, Q)) return FP8Q_ERR_SHAPE;
  if (M_tot / 128 + G >= kMaxDim) return FP8Q_ERR_SHAPE;
  // a workgroup per 128 x 128 tile of C, an expert's rounded up to eight of them
  if (!fp8q::grid_fits(8 * G * (((P / 128) * (Q / 128) + 7) / 8), 512)) return FP8Q_ERR_SHAPE;
  if (P == 0 || Q == 0) return FP8Q_OK;
  if (!c || !offsets || (M_tot > 0 && (!aq || !sa || !bq || !sb))) return FP8Q_ERR_NULL;
  if (misaligned(aq) || misaligned(sa) || misaligned(bq) || misaligned(sb) || misaligned(offsets, 4) || misaligned(c))
    return FP8Q_ERR_ALIGN;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_grouped_gemm_rowscaled(aq, sa, bq, sb, offsets, G, M_tot, P, Q, c,
                                                      out_dtype == FP8Q_OUT_F32, as_stream(stream)));
}

fp8q_status fp8q_adamw(const fp8q_adamw_tensor *tensors, int64_t count, int32_t grad_dtype, int32_t state_dtype,
                       const fp8q_adamw_hyper *hyper, void *stream) {
  if (bad_dtype(grad_dtype) || (state_dtype != FP8Q_STATE_F32 && state_dtype != FP8Q_STATE_E4M3))
    return FP8Q_ERR_DTYPE;
  if (bad_dim(count)) return FP8Q_ERR_SHAPE;
  if (!hyper || (count > 0 && !tensors)) return FP8Q_ERR_NULL;
  const fp8q_adamw_hyper &h = *hyper;
  const double numbers[] = {h.lr, h.beta1, h.beta2, h.eps, h.weight_decay, h.grad_scale};
  for (double v : numbers)
    if (!f32_number(v)) return FP8Q_ERR_VALUE;
  if (!f32_beta(h.beta1) || !f32_beta(h.beta2) || h.eps < 0 || h.step < 1) return FP8Q_ERR_VALUE;
  if (!h.scalars && (!(fabs(1.0 - h.lr * h.weight_decay) <= FLT_MAX) ||
                     !(fabs(h.lr / (1.0 - pow(h.beta1, static_cast<double>(h.step)))) <= FLT_MAX)))
    return FP8Q_ERR_VALUE;
  const bool e4m3 = state_dtype == FP8Q_STATE_E4M3;
  bool work = false;
  for (int64_t i = 0; i < count; ++i) {
    const fp8q_adamw_tensor &t = tensors[i];
    if (t.n < 0 || !fp8q::grid_fits(t.n / fp8q::kAdamwPerGroup + (t.n % fp8q::kAdamwPerGroup != 0), 256))
      return FP8Q_ERR_SHAPE;
    if (t.n == 0) continue;
    if (!t.p || !t.grad || !t.m || !t.v || (e4m3 && (!t.m_scale || !t.v_scale))) return FP8Q_ERR_NULL;
    if (misaligned(t.p) || misaligned(t.grad) || misaligned(t.m) || misaligned(t.v) || misaligned(t.p_bf16) ||
        (e4m3 && (misaligned(t.m_scale, 4) || misaligned(t.v_scale, 4))))
      return FP8Q_ERR_ALIGN;
    work = true;
  }
  if (misaligned(h.scalars, 4)) return FP8Q_ERR_ALIGN;
  if (!work) return FP8Q_OK;
  if (device_ok() != FP8Q_OK) return FP8Q_ERR_DEVICE;
  return launched(fp8q::launch_adamw(tensors, count, grad_dtype == FP8Q_OUT_F32, e4m3, h, as_stream(stream)));
}

const char *fp8q_status_string(fp8q_status status) {
  switch (status) {
    case FP8Q_OK: return "ok";
    case FP8Q_ERR_NULL: return "null pointer argument";
    case FP8Q_ERR_SHAPE: return "invalid shape (negative, K/N (or M for the dual quantizer) not a multiple of 128, G < 1, or too large)";
    case FP8Q_ERR_ALIGN: return "misaligned pointer (16-byte alignment required; offsets 4-byte)";
    case FP8Q_ERR_DTYPE: return "invalid dtype argument";
    case FP8Q_ERR_DEVICE: return "no usable HIP device";
    case FP8Q_ERR_LAUNCH: return "kernel launch failed";
    case FP8Q_ERR_OFFSETS: return "grouped GEMM offsets invalid (offsets[0] != 0, decreasing, or offsets[G] != M_tot)";
    case FP8Q_ERR_VALUE: return "hyperparameter out of range (not a finite FP32 number, beta outside [0, 1), eps < 0, step < 1, or lr / (1 - beta1^step) or lr * weight_decay past FP32)";
    default: return "unknown status";
  }
}

int32_t fp8q_abi_version(void) { return FP8Q_ABI_VERSION; }

}  // extern "C"
