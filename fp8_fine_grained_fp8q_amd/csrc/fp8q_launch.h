// Internal launchers of libfp8q (host side).  Arguments are validated by the C ABI layer
// before any of these is called; each returns the launch's hipError_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q.h"

namespace fp8q {

// HIP supports fewer than 2^32 threads per dimension of a grid.
inline bool grid_fits(int64_t groups, int64_t threads) { return groups < (int64_t(1) << 32) / threads; }

// Compute units of the current device (cached per device; 256 if the query fails).
int device_cu_count();

hipError_t launch_quant_act(const uint16_t *x, int64_t M, int64_t K, uint8_t *xq, float *sa,
                            hipStream_t stream);

// launch_quant_act and launch_quant_w (no W^T) for X[M][K] and W[G][N][K] in one launch.
hipError_t launch_quant_act_w(const uint16_t *x, int64_t M, uint8_t *xq, float *sa, const uint16_t *w, int64_t G,
                              int64_t N, uint8_t *wq, float *sb, int64_t K, hipStream_t stream);

// wqt / sbt (W^T codes and block scales) are written too unless wqt is null.
hipError_t launch_quant_w(const uint16_t *w, int64_t G, int64_t N, int64_t K, uint8_t *wq, float *sb,
                          uint8_t *wqt, float *sbt, hipStream_t stream);

// Both orientations of X[M][K] (M % 128 == 0): 1x128 tiles along K (xq, sa as above)
// and 128x1 tiles along M, codes channel-major xqt[K][M], scales sat[M/128][K].
hipError_t launch_quant_act_dual(const uint16_t *x, int64_t M, int64_t K, uint8_t *xq, float *sa,
                                 uint8_t *xqt, float *sat, hipStream_t stream);

// h = SiLU(g) * u of gu[M][2I] (g left half, u right half), quantized in 1x128 tiles.
hipError_t launch_swiglu_quant_act(const uint16_t *gu, int64_t M, int64_t I, uint8_t *xq, float *sa,
                                   hipStream_t stream);

// One scale for n BF16 values (n % 8 == 0): from the tensor's amax (scale_in null) or the
// caller's scale; stats[0..2] = amax bits, saturated count, scale bits.
hipError_t launch_quant_per_tensor(const uint16_t *x, int64_t n, const float *scale_in, uint8_t *q,
                                   uint32_t *stats, hipStream_t stream);

hipError_t launch_gemm(const uint8_t *xq, const float *sa, const uint8_t *wq, const float *sb,
                       int64_t M, int64_t N, int64_t K, void *c, bool out_f32, hipStream_t stream);

// C = dequant(aq, sa) dequant(bq, sb)^T, both with 1x128 row scales ([K/128][rows]).
hipError_t launch_gemm_rowscaled(const uint8_t *aq, const float *sa, const uint8_t *bq, const float *sb,
                                 int64_t M, int64_t N, int64_t K, void *c, bool out_f32, hipStream_t stream);

// Debug check of grouped-GEMM offsets (offsets[0] == 0, non-decreasing, offsets[G] == M_tot)
// on `stream`; waits for the stream and sets *bad.
hipError_t check_grouped_offsets(const int32_t *offsets, int64_t G, int64_t M_tot, hipStream_t stream, bool *bad);

hipError_t launch_grouped_gemm(const uint8_t *xq, const float *sa, const uint8_t *wq, const float *sb,
                               const int32_t *offsets, int64_t G, int64_t M_tot, int64_t N, int64_t K,
                               void *c, bool out_f32, hipStream_t stream);

// Expert-parallel dispatch on the GPU owning experts [e_begin, e_begin + E): route the
// top-k ids [T][k] (offsets [E+1], token_row [T][k], row_token [cap]) and pack the routed
// rows' codes xq [T][K] / scales sa [K/128][T] into xq_s [cap][K] / sa_s [K/128][cap].
hipError_t launch_moe_dispatch(const int32_t *ids, int64_t T, int64_t k, int64_t e_begin, int64_t E,
                               const uint8_t *xq, const float *sa, int64_t K, int64_t cap, uint8_t *xq_s,
                               float *sa_s, int32_t *offsets, int32_t *token_row, int32_t *row_token,
                               hipStream_t stream);

// y[t] = sum over slots s with 0 <= token_row[t][s] < cap of w[t][s] * out[token_row[t][s]].
hipError_t launch_moe_combine(const void *out, bool in_f32, int64_t cap, int64_t N, const int32_t *token_row,
                              const float *w, int64_t T, int64_t k, void *y, bool out_f32, hipStream_t stream);

// Workgroups of 256 threads of the copy in launch_moe_sort (the routing's fit for every T * k < 2^31).
int64_t moe_sort_groups(int64_t T, int64_t k, bool f32, int64_t H);

// The dispatch's routing with values in place of codes: xs[token_row[t][s]] = x[t], rows of H
// BF16 or FP32 values.
hipError_t launch_moe_sort(const int32_t *ids, int64_t T, int64_t k, int64_t e_begin, int64_t E, const void *x,
                           bool f32, int64_t H, int64_t cap, void *xs, int32_t *offsets, int32_t *token_row,
                           int32_t *row_token, hipStream_t stream);

// dx[t] = sum over slots s with 0 <= token_row[t][s] < cap of dxs[token_row[t][s]].
hipError_t launch_moe_sort_backward(const void *dxs, bool in_f32, int64_t cap, int64_t H, const int32_t *token_row,
                                    int64_t T, int64_t k, void *dx, bool out_f32, hipStream_t stream);

// Gradients of launch_moe_combine: dout[row] = w[t][s] * dy[t], dw[t][s] = <out[row], dy[t]>.
hipError_t launch_moe_combine_backward(const void *dy, bool dy_f32, const void *out, bool f32, int64_t cap, int64_t N,
                                       const int32_t *token_row, const float *w, int64_t T, int64_t k, void *dout,
                                       float *dw, hipStream_t stream);

// dgu = gradient of h = SiLU(g) * u (layout of gu); h itself too unless null.
hipError_t launch_swiglu_backward(const uint16_t *gu, const void *dh, bool dh_f32, int64_t M, int64_t I,
                                  uint16_t *dgu, uint16_t *h, hipStream_t stream);

// Token tiles of expert-sorted rows, none across two experts: xqt[B][K][128], sat[B][K], B =
// M / 128 + G; the rows' 1x128 codes xq[M][K], sa[K/128][M] too unless xq is null.
hipError_t launch_quant_act_grouped(const uint16_t *x, const int32_t *offsets, int64_t G, int64_t M, int64_t K,
                                    uint8_t *xq, float *sa, uint8_t *xqt, float *sat,
                                    hipStream_t stream);

// C[g] = dequant(aq, sa) dequant(bq, sb)^T over expert g's token tiles.
hipError_t launch_grouped_gemm_rowscaled(const uint8_t *aq, const float *sa, const uint8_t *bq, const float *sb,
                                         const int32_t *offsets, int64_t G, int64_t M, int64_t P, int64_t Q,
                                          void *c, bool out_f32, hipStream_t stream);

constexpr int64_t kAdamwPerGroup = 2048;  // elements of a workgroup of 256 threads

// One AdamW step over `count` tensors (host array).
hipError_t launch_adamw(const fp8q_adamw_tensor *tensors, int64_t count, bool grad_f32, bool e4m3,
                        const fp8q_adamw_hyper &hyper, hipStream_t stream);

constexpr int64_t kMaxNormWidth = 16384;  // columns: 1024 threads of 16
constexpr int64_t kNormGroups = 256;      // the most workgroups that layer norm's gradient leaves sums of

// Workgroups of launch_layer_norm_backward for T rows; its `part` holds 2 H floats for each (H without db).
int64_t norm_backward_groups(int64_t T);

// y = (x - mean) rstd w + b of rows of H values (center false: RMS norm, mean not written); b may be null.
hipError_t launch_layer_norm(const void *x, bool x_f32, const float *w, const float *b, int64_t T, int64_t H, float eps,
                             bool center, void *y, bool out_f32, float *mean, float *rstd, hipStream_t stream);

// dx, dw and db (unless null) of launch_layer_norm; mean null: RMS norm.
hipError_t launch_layer_norm_backward(const void *dy, bool dy_f32, const void *x, bool x_f32, const float *w,
                                      const float *mean, const float *rstd, int64_t T, int64_t H, void *dx, bool out_f32,
                                      float *dw, float *db, float *part, hipStream_t stream);

constexpr int kMaxTopK = 64;
constexpr int64_t kMaxSequences = 65535;  // the second dimension of a grid
constexpr int64_t kRouteGroups = 256;     // the most workgroups per sequence of the router

// Bytes of launch_moe_route's workspace (16-byte aligned).
int64_t moe_route_workspace(int64_t B, int64_t S, int64_t E);

// Top-k experts of B sequences of S tokens from their logits [B][S][E], gating weights, counts [B][E] and
// the balance loss with its slope [B][E].
hipError_t launch_moe_route(const void *logits, bool f32, int64_t B, int64_t S, int64_t E, int64_t k, const float *bias,
                            const uint8_t *valid, bool softmax, bool normalize, float scale, double balance, int32_t *ids,
                            float *w, int32_t *counts, float *loss, float *slope, void *workspace, hipStream_t stream);

// Gradient of the weights (dw) and of the loss (dloss, 1 if null) by the logits.
hipError_t launch_moe_route_backward(const void *logits, bool f32, int64_t B, int64_t S, int64_t E, int64_t k,
                                     const int32_t *ids, const float *w, const float *dw, const float *slope,
                                     const float *dloss, bool softmax, bool normalize, float scale, void *dlogits,
                                     bool out_f32, hipStream_t stream);

// Bytes of the workspace of the two calls below (16-byte aligned), and whether their launches fit HIP's grids.
int64_t muon_workspace(int64_t G, int64_t P, int64_t Q);
bool muon_grids_fit(int64_t G, int64_t P, int64_t Q);

// BF16 matrices [G][P][Q] with the singular vectors of x and singular values near one.
hipError_t launch_orthogonalize(const void *x, bool f32, int64_t G, int64_t P, int64_t Q, const fp8q_newton_schulz &ns,
                                uint16_t *out, void *workspace, hipStream_t stream);

// A Muon step on G matrices: momentum, the update made orthogonal, the parameter (and its BF16 copy unless null).
hipError_t launch_muon(float *param, const void *grad, bool f32, float *momentum, int64_t G, int64_t P, int64_t Q,
                       const fp8q_muon_hyper &hyper, uint16_t *copy, void *workspace, hipStream_t stream);

}  // namespace fp8q
