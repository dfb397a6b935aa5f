// Gradient of SwiGLU, h = SiLU(g) * u, the activation between the expert projections
// (risenshineclean.com page, section 2, on the expert FFN; the pages do not name the
// activation, SwiGLU is the reading taken by the forward kernel too), for gfx950.
//
// With s = 1 / (1 + e^-g):  du = dh * g s,  dg = dh * u * s (1 + g (1 - s)),  h = g s u.
// s and 1 - s are both formed from e^-|g| (no overflow for any g, no cancellation in 1 - s)
// with the hardware reciprocal (one ulp), all in FP32 with one rounding at the end.  Products are
// ordered so that none overflows in between: g u first would make inf * 0 of a large u beside a
// closed gate.
//
// Bound by HBM: 4 bytes of gu and 2 or 4 of dh in, 4 bytes of dgu out per element of h, and
// 2 more for h itself, which the down projection's weight gradient contracts with and the
// forward pass has kept as codes in the other orientation only.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

template <bool kDhF32>
__global__ __launch_bounds__(256) void swiglu_backward_kernel(const uint16_t *__restrict__ gu,
                                                              const void *__restrict__ dh, uint64_t chunks,
                                                              uint32_t per_row, uint16_t *__restrict__ dgu,
                                                              uint16_t *__restrict__ h) {
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x;  // 8 columns of h
  if (i >= chunks) return;
  const uint64_t row = chunks <= 0xffffffffu ? static_cast<uint32_t>(i) / per_row : i / per_row;
  const int64_t at_g = static_cast<int64_t>(i + row * per_row) * 8;  // row * 2I + column
  const int64_t at_u = at_g + static_cast<int64_t>(per_row) * 8;
  float g[8], u[8], d[8];
  load8<false>(gu, at_g, g);
  load8<false>(gu, at_u, u);
  load8<kDhF32>(dh, static_cast<int64_t>(i) * 8, d);
  float dg[8], du[8], hv[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = expf(-fabsf(g[e]));
    const float r = __builtin_amdgcn_rcpf(1.0f + t);
    const float s = (g[e] >= 0.0f ? 1.0f : t) * r;  // sigma(g)
    const float c = (g[e] >= 0.0f ? t : 1.0f) * r;  // 1 - sigma(g)
    const float silu = g[e] * s, slope = s * __builtin_fmaf(g[e], c, 1.0f);  // |slope| < 1.1
    hv[e] = silu * u[e];
    du[e] = silu * d[e];
    // the larger of d and u meets the slope first, halved: no overflow but the result's own
    const bool less = fabsf(d[e]) < fabsf(u[e]);
    dg[e] = (0.5f * slope) * (less ? u[e] : d[e]) * (less ? d[e] : u[e]) * 2.0f;
  }
  store8<false>(dgu, at_g, dg);
  store8<false>(dgu, at_u, du);
  if (h != nullptr) store8<false>(h, static_cast<int64_t>(i) * 8, hv);
}

hipError_t launch_swiglu_backward(const uint16_t *gu, const void *dh, bool dh_f32, int64_t M, int64_t I, uint16_t *dgu,
                                  uint16_t *h, hipStream_t stream) {
  const int64_t chunks = M * (I / 8), blocks = (chunks + 255) / 256;
  const dim3 grid(static_cast<uint32_t>(blocks)), block(256);
  const uint64_t n = static_cast<uint64_t>(chunks);
  const uint32_t per_row = static_cast<uint32_t>(I / 8);
  if (dh_f32)
    hipLaunchKernelGGL(swiglu_backward_kernel<true>, grid, block, 0, stream, gu, dh, n, per_row, dgu, h);
  else
    hipLaunchKernelGGL(swiglu_backward_kernel<false>, grid, block, 0, stream, gu, dh, n, per_row, dgu, h);
  return hipGetLastError();
}

}  // namespace fp8q
