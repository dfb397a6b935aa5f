// AdamW over many tensors in one launch, states in FP32 or in E4M3, for gfx950.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps),  g scaled first.
//
// E4M3 states hold m and r = sqrt(v) as codes with one FP32 scale amax / 448 per 128
// consecutive elements, the activation quantizer's tile and rounding (codingmall.com page,
// sections "Dinh luong hat min", "Dinh dang E4M3 hop nhat": one FP8 format, small groups;
// that the optimizer states take it is this library's reading).  r rather than v: E4M3
// reaches from 448 down to 2^-9, 18 binary orders, and the root needs half as many as v.  A
// nonzero r never becomes code 0 but the smallest code: with v = 0 and m != 0 the next step
// would divide by eps alone.  The new p uses m and v before they are rounded to E4M3.
//
// Bound by HBM: 28 bytes per element with FP32 states and gradients, 16.1 with E4M3 states
// (p 4 + 4, g 4, m and r 1 + 1 each, two scales per 128).  Each thread takes 8 consecutive
// elements, so a tile of 128 is one 16-lane DPP row; a workgroup takes 2048.  The tensors'
// addresses and sizes travel in the kernel arguments (no table in device memory to fill,
// nothing to wait for): 76 or 58 of them per launch.
//
// Every operation is rounded to FP32 by itself (no contraction), in the order above, so the
// result is the same as that of separate FP32 operations, bit for bit.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "fp8q.h"
#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

constexpr int64_t kPerBlock = kAdamwPerGroup;

// The descriptors of a launch: as many as its 4 KB of kernel arguments hold.
struct AdamE4M3 {
  float *p;
  const void *grad;
  void *m, *v;
  float *m_scale, *v_scale;
  uint16_t *p_bf16;
  int64_t n;
};
struct AdamF32 {
  float *p;
  const void *grad;
  void *m, *v;
  uint16_t *p_bf16;
  int64_t n;
};

template <bool kE4M3>
struct AdamTable {
  using Tensor = std::conditional_t<kE4M3, AdamE4M3, AdamF32>;
  static constexpr int kMax = kE4M3 ? 58 : 76;
  Tensor t[kMax];
  uint32_t first[kMax + 1];  // first workgroup of each tensor, and the end
  int count;
};

struct AdamHyper {
  float b1, c1, b2, c2;  // beta and 1 - beta
  float eps, wd;
  float decay, step, root;  // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float grad_scale;
  const float *scalars;  // device {lr, 1 - b1^t, 1 - b2^t, grad_scale} in place of the host's, or null
};

static_assert(sizeof(AdamTable<true>) + sizeof(AdamHyper) <= 4096, "kernel arguments");
static_assert(sizeof(AdamTable<false>) + sizeof(AdamHyper) <= 4096, "kernel arguments");

// Values [at, at + 8) of an array of n, zeros past its end.
template <bool kF32>
__device__ __forceinline__ void load8_tail(const void *p, int64_t at, int64_t n, float (&v)[8]) {
  if (at + 8 <= n) {
    load8<kF32>(p, at, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.0f;
    if (at + i < n)
      v[i] = kF32 ? static_cast<const float *>(p)[at + i] : bf16_lo(static_cast<const uint16_t *>(p)[at + i]);
  }
}

template <bool kF32>
__device__ __forceinline__ void store8_tail(void *p, int64_t at, int64_t n, const float (&v)[8]) {
  if (at + 8 <= n) {
    store8<kF32>(p, at, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (at + i >= n) break;
    if (kF32)
      static_cast<float *>(p)[at + i] = v[i];
    else
      static_cast<uint16_t *>(p)[at + i] = static_cast<uint16_t>(pack2_bf16(v[i], 0.0f));
  }
}

__device__ __forceinline__ uint2 load_codes(const uint8_t *p, int64_t at, int64_t n) {
  if (at + 8 <= n) return *reinterpret_cast<const uint2 *>(p + at);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + i < n) w[i >> 2] |= static_cast<uint32_t>(p[at + i]) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(uint8_t *p, int64_t at, int64_t n, uint2 q) {
  if (at + 8 <= n) {
    *reinterpret_cast<uint2 *>(p + at) = q;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + i < n) p[at + i] = static_cast<uint8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
}

__device__ __forceinline__ void decode8(uint2 q, float s, float (&v)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), true);
    v[4 * i] = lo.x * s;
    v[4 * i + 1] = lo.y * s;
    v[4 * i + 2] = hi.x * s;
    v[4 * i + 3] = hi.y * s;
  }
}

// Codes and scale of one 16-lane tile of FP32 values; kRoot: the values are non-negative and
// a nonzero one gets a nonzero code.
template <bool kRoot>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float &s) {
  float a = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  s = row16_max(a) / kE4M3Max;
  const GroupDiv dv(s);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = dv.mode == 1 ? dv.fast(x[i]) : (dv.mode == 2 ? x[i] / dv.s : x[i]);
    if (kRoot) y[i] = fmaxf(y[i], x[i] > 0.0f ? 0x1p-9f : 0.0f);
  }
  return make_uint2(pack4_e4m3(y[0], y[1], y[2], y[3]), pack4_e4m3(y[4], y[5], y[6], y[7]));
}

template <bool kE4M3, bool kGradF32>
__global__ __launch_bounds__(256) void adamw_kernel(const AdamTable<kE4M3> table, const AdamHyper hy) {
#pragma clang fp contract(off)
  int lo = 0, hi = table.count - 1;  // the last tensor whose first workgroup is not behind this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table.first[mid] <= blockIdx.x)
      lo = mid;
    else
      hi = mid - 1;
  }
  const auto &t = table.t[lo];
  const int64_t n = t.n;
  const int64_t at = (static_cast<int64_t>(blockIdx.x - table.first[lo]) * 256 + threadIdx.x) * 8;
  float decay = hy.decay, step = hy.step, root = hy.root, scale = hy.grad_scale;
  if (hy.scalars != nullptr) {
    const float lr = hy.scalars[0];
    decay = 1.0f - lr * hy.wd;
    step = lr / hy.scalars[1];
    root = 1.0f / sqrtf(hy.scalars[2]);
    scale = hy.scalars[3];
  }
  if (!kE4M3 && at >= n) return;
  if (kE4M3 && (at & ~int64_t(127)) >= n) return;  // whole 16-lane tiles leave together

  float p[8], g[8], m[8], v[8];
  load8_tail<true>(t.p, at, n, p);
  load8_tail<kGradF32>(t.grad, at, n, g);
  if constexpr (kE4M3) {
    const int64_t tile = at >> 7;
    decode8(load_codes(static_cast<const uint8_t *>(t.m), at, n), t.m_scale[tile], m);
    decode8(load_codes(static_cast<const uint8_t *>(t.v), at, n), t.v_scale[tile], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * v[i];
  } else {
    load8_tail<true>(t.m, at, n, m);
    load8_tail<true>(t.v, at, n, v);
  }
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = g[i] * scale;
    m[i] = m[i] * hy.b1 + gi * hy.c1;
    v[i] = v[i] * hy.b2 + (gi * hy.c2) * gi;
    r[i] = sqrtf(v[i]);
    p[i] = p[i] * decay - (m[i] / (r[i] * root + hy.eps)) * step;
  }
  store8_tail<true>(t.p, at, n, p);
  if (t.p_bf16 != nullptr) store8_tail<false>(t.p_bf16, at, n, p);
  if constexpr (kE4M3) {
    // elements past the end are zeros in every array, so they change no maximum
    float ms, vs;
    const uint2 mq = encode8<false>(m, ms), vq = encode8<true>(r, vs);
    store_codes(static_cast<uint8_t *>(t.m), at, n, mq);
    store_codes(static_cast<uint8_t *>(t.v), at, n, vq);
    if ((threadIdx.x & 15) == 0) {
      t.m_scale[at >> 7] = ms;
      t.v_scale[at >> 7] = vs;
    }
  } else {
    store8_tail<true>(t.m, at, n, m);
    store8_tail<true>(t.v, at, n, v);
  }
}

namespace {

AdamE4M3 descriptor(const fp8q_adamw_tensor &t, const AdamE4M3 *) {
  return {t.p, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.p_bf16, t.n};
}
AdamF32 descriptor(const fp8q_adamw_tensor &t, const AdamF32 *) { return {t.p, t.grad, t.m, t.v, t.p_bf16, t.n}; }

template <bool kE4M3>
hipError_t launch_batches(const fp8q_adamw_tensor *tensors, int64_t count, bool grad_f32, const AdamHyper &hy,
                          hipStream_t stream) {
  for (int64_t i = 0; i < count;) {
    AdamTable<kE4M3> table;
    table.count = 0;
    int64_t blocks = 0;
    for (; i < count && table.count < AdamTable<kE4M3>::kMax; ++i) {
      const int64_t b = (tensors[i].n + kPerBlock - 1) / kPerBlock;
      if (b == 0) continue;
      if (!grid_fits(blocks + b, 256)) break;  // the caller has checked that one tensor fits
      table.t[table.count] = descriptor(tensors[i], table.t);
      table.first[table.count++] = static_cast<uint32_t>(blocks);
      blocks += b;
    }
    if (table.count == 0) continue;
    table.first[table.count] = static_cast<uint32_t>(blocks);
    const dim3 grid(static_cast<uint32_t>(blocks)), block(256);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, table, hy); };
    grad_f32 ? go(adamw_kernel<kE4M3, true>) : go(adamw_kernel<kE4M3, false>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_adamw(const fp8q_adamw_tensor *tensors, int64_t count, bool grad_f32, bool e4m3,
                        const fp8q_adamw_hyper &h, hipStream_t stream) {
  AdamHyper hy;
  hy.b1 = static_cast<float>(h.beta1);
  hy.c1 = static_cast<float>(1.0 - h.beta1);
  hy.b2 = static_cast<float>(h.beta2);
  hy.c2 = static_cast<float>(1.0 - h.beta2);
  hy.eps = static_cast<float>(h.eps);
  hy.wd = static_cast<float>(h.weight_decay);
  hy.decay = static_cast<float>(1.0 - h.lr * h.weight_decay);
  hy.step = static_cast<float>(h.lr / (1.0 - pow(h.beta1, static_cast<double>(h.step))));
  hy.root = static_cast<float>(1.0 / sqrt(1.0 - pow(h.beta2, static_cast<double>(h.step))));
  hy.grad_scale = static_cast<float>(h.grad_scale);
  hy.scalars = h.scalars;
  return e4m3 ? launch_batches<true>(tensors, count, grad_f32, hy, stream)
              : launch_batches<false>(tensors, count, grad_f32, hy, stream);
}

}  // namespace fp8q
