// Layer norm and RMS norm of rows and their gradients, for gfx950: the norm whose output the
// activation quantizer and the router read.
//
//   mean = sum x / H (0 for RMS norm),  rstd = 1 / sqrt(sum (x - mean)^2 / H + eps),
//   h = (x - mean) rstd,  y = h w + b,
//   g = dy w,  dx = rstd (g - sum g / H - h sum g h / H)  (RMS norm: without sum g),
//   dw = sum over rows of dy h,  db = sum over rows of dy.
//
// Bound by HBM from about 4096 columns on: x in and y out, or x and dy in and dx out.  A row stays in the registers of
// one workgroup (8 columns per thread, or 16 of more than 8192), so x is read once and the squares are those
// of x - mean.  Workgroups take every gridDim.x-th row and load the next one before they sum this
// one; the weights stay in registers too.  All sums are FP32, in an order that depends on the sizes
// only, with one rounding of each result.
//
// 16384 x 7168 from FP32 to BF16: 133 us, 5.3 TB/s (a copy kernel of this card's best 6.16 TB/s: 114).  Gradient of
// 8192 x 7168 in BF16: 61 us, 5.7 TB/s (with one row on its way and cached loads 80), and 5 us for the sums.
// Narrow rows are bound by the steps of a workgroup's rows, one row at a time (whole calls, BF16, copy's floor in
// brackets): 8192 x 1024 12 us (5) and gradient 28 us (8), 8192 x 256 11 (1.4) and 20 (2), 2^20 x 128 293 (87) and 1860
// (131): the gradient has kNormGroups workgroups whatever their size, of one wave each up to 512 columns.  Rows above 8192
// cost the gradient registers: 16 columns per thread of x, dy, their next rows, weights and sums spill 56 to 268 bytes of
// scratch per thread; 4096 x 16384 105 us in BF16 (65), 402 in FP32 (131).
//
// dw and db: every workgroup of the backward kernel keeps its rows' sums in registers and leaves
// them in the workspace, 4 H bytes each; a second kernel adds up at most kNormGroups of them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

namespace {


// Eight values as they lie in memory, read once.
template <bool kF32>
struct Raw8 {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const void *p, int64_t off) {
    if (kF32) {
      const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + off);
      lo = load16_stream(q);
      hi = load16_stream(q + 1);
    } else {
      lo = load16_stream(static_cast<const uint16_t *>(p) + off);
    }
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w};
    if (kF32) {
      const uint32_t b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(a[i]);
        v[2 * i + 1] = bf16_hi(a[i]);
      }
    }
  }
};

// Sum over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x128, 0xf, 0xf, false);  // row_ror:8
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x124, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x122, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x121, 0xf, 0xf, false);
  return (lane_f32(v, 0) + lane_f32(v, 16)) + (lane_f32(v, 32) + lane_f32(v, 48));
}

// LDS of the workgroup's sums: two places in turn, so that one barrier per sum suffices.
struct Sums {
  float2 part[2][16];
};

// The sums of a and b over the workgroup, in every thread.  The barrier waits for LDS only: the next
// row's loads stay in flight.
__device__ __forceinline__ float2 group_sum(float a, float b, Sums &s, int &turn) {
  const int waves = blockDim.x >> 6;
  a = wave_sum(a);
  b = wave_sum(b);
  if (waves == 1) return make_float2(a, b);
  if ((threadIdx.x & 63) == 0) s.part[turn][threadIdx.x >> 6] = make_float2(a, b);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  float2 t = make_float2(0.0f, 0.0f);
  for (int w = 0; w < waves; ++w) {
    const float2 p = s.part[turn][w];
    t.x += p.x;
    t.y += p.y;
  }
  turn ^= 1;
  return t;
}

template <int kNC, bool kXF32, bool kOutF32, bool kCenter>
__global__ __launch_bounds__(1024) void layer_norm_kernel(const void *__restrict__ x, const float *__restrict__ w,
                                                          const float *__restrict__ b, int64_t T, int chunks, float eps,
                                                          void *__restrict__ y, float *__restrict__ mean,
                                                          float *__restrict__ rstd) {
  __shared__ Sums sums;
  int turn = 0;
  const int64_t H = static_cast<int64_t>(chunks) * 8;
  const float n = static_cast<float>(H);
  float wv[kNC][8], bv[kNC][8];
  Raw8<kXF32> raw[kNC] = {};
  int64_t row = blockIdx.x;
#pragma unroll
  for (int j = 0; j < kNC; ++j) {
    const int c = threadIdx.x + j * blockDim.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[j][i] = bv[j][i] = 0.0f;
    if (c < chunks) {
      raw[j].load(x, row * H + c * 8);
      load8<true>(w, c * 8, wv[j]);
      if (b != nullptr) load8<true>(b, c * 8, bv[j]);
    }
  }
  for (; row < T; row += gridDim.x) {
    float v[kNC][8];
#pragma unroll
    for (int j = 0; j < kNC; ++j) raw[j].unpack(v[j]);  // zeros past the row's end
    const int64_t next = row + gridDim.x;
    if (next < T) {
#pragma unroll
      for (int j = 0; j < kNC; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        if (c < chunks) raw[j].load(x, next * H + c * 8);
      }
    }
    float m = 0.0f;
    if (kCenter) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < kNC; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[j][i];
      m = group_sum(s, 0.0f, sums, turn).x / n;
#pragma unroll
      for (int j = 0; j < kNC; ++j)
        if (static_cast<int>(threadIdx.x + j * blockDim.x) < chunks)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] -= m;
    }
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < kNC; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) q = __builtin_fmaf(v[j][i], v[j][i], q);
    const float r = 1.0f / sqrtf(group_sum(q, 0.0f, sums, turn).x / n + eps);
    if (threadIdx.x == 0) {
      if (kCenter) mean[row] = m;
      rstd[row] = r;
    }
#pragma unroll
    for (int j = 0; j < kNC; ++j) {
      const int c = threadIdx.x + j * blockDim.x;
      if (c >= chunks) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = __builtin_fmaf(v[j][i] * r, wv[j][i], bv[j][i]);
      store8<kOutF32>(y, row * H + c * 8, v[j]);
    }
  }
}

template <int kNC, bool kXF32, bool kDyF32, bool kOutF32, bool kCenter>
__global__ __launch_bounds__(1024) void layer_norm_backward_kernel(
    const void *__restrict__ dy, const void *__restrict__ x, const float *__restrict__ w, const float *__restrict__ mean,
    const float *__restrict__ rstd, int64_t T, int chunks, bool want_bias, void *__restrict__ dx,
    float *__restrict__ part) {
  __shared__ Sums sums;
  int turn = 0;
  const int64_t H = static_cast<int64_t>(chunks) * 8;
  const float over_n = 1.0f / static_cast<float>(H);
  float wv[kNC][8], dw[kNC][8], db[kNC][8];
  // Two rows are on their way, in places that take turns.
  Raw8<kXF32> raw_x[2][kNC] = {};
  Raw8<kDyF32> raw_d[2][kNC] = {};
  float mean_of[2] = {}, rstd_of[2] = {};
  auto load = [&](int64_t row, auto place) {
    constexpr int kAt = decltype(place)::value;
    if (row >= T) return;
    if (kCenter) mean_of[kAt] = mean[row];
    rstd_of[kAt] = rstd[row];
#pragma unroll
    for (int j = 0; j < kNC; ++j) {
      const int c = threadIdx.x + j * blockDim.x;
      if (c < chunks) {
        raw_x[kAt][j].load(x, row * H + c * 8);
        raw_d[kAt][j].load(dy, row * H + c * 8);
      }
    }
  };
  using First = std::integral_constant<int, 0>;
  using Second = std::integral_constant<int, 1>;
  const int64_t stride = gridDim.x;
  load(blockIdx.x, First{});
  load(blockIdx.x + stride, Second{});
#pragma unroll
  for (int j = 0; j < kNC; ++j) {
    const int c = threadIdx.x + j * blockDim.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[j][i] = dw[j][i] = db[j][i] = 0.0f;
    if (c < chunks) load8<true>(w, c * 8, wv[j]);
  }
  auto step = [&](int64_t row, auto place) {
    constexpr int kAt = decltype(place)::value;
    const float m = mean_of[kAt], r = rstd_of[kAt];
    float h[kNC][8], d[kNC][8];
#pragma unroll
    for (int j = 0; j < kNC; ++j) {
      raw_x[kAt][j].unpack(h[j]);
      raw_d[kAt][j].unpack(d[j]);  // zeros past the row's end
    }
    load(row + 2 * stride, place);
    float s = 0.0f, t = 0.0f;  // sums of g h and of g
#pragma unroll
    for (int j = 0; j < kNC; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[j][i] = (kCenter ? h[j][i] - m : h[j][i]) * r;
        dw[j][i] = __builtin_fmaf(d[j][i], h[j][i], dw[j][i]);
        db[j][i] += d[j][i];
        d[j][i] *= wv[j][i];
        s = __builtin_fmaf(d[j][i], h[j][i], s);
        t += d[j][i];
      }
    const float2 all = group_sum(s, kCenter ? t : 0.0f, sums, turn);
    s = all.x * over_n;
    t = all.y * over_n;
#pragma unroll
    for (int j = 0; j < kNC; ++j) {
      const int c = threadIdx.x + j * blockDim.x;
      if (c >= chunks) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = kCenter ? d[j][i] - t : d[j][i];
        d[j][i] = r * __builtin_fmaf(-h[j][i], s, e);
      }
      store8<kOutF32>(dx, row * H + c * 8, d[j]);
    }
  };
  for (int64_t row = blockIdx.x; row < T; row += 2 * stride) {
    step(row, First{});
    if (row + stride < T) step(row + stride, Second{});
  }
  float *mine = part + static_cast<int64_t>(blockIdx.x) * H;
  float *bias = part + (static_cast<int64_t>(gridDim.x) + blockIdx.x) * H;
#pragma unroll
  for (int j = 0; j < kNC; ++j) {
    const int c = threadIdx.x + j * blockDim.x;
    if (c >= chunks) break;
    store8<true>(mine, c * 8, dw[j]);
    if (want_bias) store8<true>(bias, c * 8, db[j]);
  }
}

// out[c] = sum over `groups` rows of part[.][c], for 64 columns by 16 slices of the rows; blockIdx.y: dw, db.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float *__restrict__ part, int groups, int H,
                                                        float *__restrict__ dw, float *__restrict__ db) {
  __shared__ float slices[16][64];
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float *p = part + static_cast<int64_t>(blockIdx.y) * groups * H;
  float s = 0.0f;
  if (c < H) {
#pragma unroll 4
    for (int g = slice; g < groups; g += 16) s += p[static_cast<int64_t>(g) * H + c];
  }
  slices[slice][lane] = s;
  __syncthreads();
  if (slice != 0 || c >= H) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) s += slices[k][lane];
  (blockIdx.y == 0 ? dw : db)[c] = s;
}

// Chunks of 8 columns per thread, and threads for them.
int norm_chunks(int64_t H) { return H <= 8192 ? 1 : 2; }
int norm_threads(int64_t H) {
  const int64_t wave = 64 * norm_chunks(H);
  return static_cast<int>((H / 8 + wave - 1) / wave * 64);
}

// bool arguments as template parameters: with(f, a, b, ...) calls f(true_or_false_type, ...).
template <class F>
hipError_t with(F f) {
  return f();
}
template <class F, class... Rest>
hipError_t with(F f, bool first, Rest... rest) {
  return first ? with([=](auto... more) { return f(std::integral_constant<bool, true>{}, more...); }, rest...)
               : with([=](auto... more) { return f(std::integral_constant<bool, false>{}, more...); }, rest...);
}

}  // namespace

int64_t norm_backward_groups(int64_t T) {
  const int64_t groups = (T + 3) / 4;
  return groups < kNormGroups ? groups : kNormGroups;
}

hipError_t launch_layer_norm(const void *x, bool x_f32, const float *w, const float *b, int64_t T, int64_t H, float eps,
                             bool center, void *y, bool out_f32, float *mean, float *rstd, hipStream_t stream) {
  const int threads = norm_threads(H);
  // Two workgroups of 14 waves on a CU: 16384 x 7168 of FP32 into BF16 132 us (5.3 TB/s), one 161, four by turns 154.
  const int64_t resident = static_cast<int64_t>(device_cu_count()) * (2048 / threads);
  const dim3 grid(static_cast<uint32_t>(T < resident ? T : resident)), block(threads);
  return with(
      [=](auto one, auto xf, auto of, auto ce) {
        hipLaunchKernelGGL((layer_norm_kernel<one.value ? 1 : 2, xf.value, of.value, ce.value>), grid, block, 0, stream, x, w, b, T,
                           static_cast<int>(H / 8), eps, y, mean, rstd);
        return hipGetLastError();
      },
      norm_chunks(H) == 1, x_f32, out_f32, center);
}

hipError_t launch_layer_norm_backward(const void *dy, bool dy_f32, const void *x, bool x_f32, const float *w,
                                      const float *mean, const float *rstd, int64_t T, int64_t H, void *dx, bool out_f32,
                                      float *dw, float *db, float *part, hipStream_t stream) {
  const int groups = static_cast<int>(norm_backward_groups(T));
  if (groups > 0) {
    const dim3 grid(groups), block(norm_threads(H));
    const hipError_t e = with(
        [=](auto one, auto xf, auto df, auto of, auto ce) {
          hipLaunchKernelGGL((layer_norm_backward_kernel<one.value ? 1 : 2, xf.value, df.value, of.value, ce.value>), grid, block, 0, stream,
                             dy, x, w, mean, rstd, T, static_cast<int>(H / 8), db != nullptr, dx, part);
          return hipGetLastError();
        },
        norm_chunks(H) == 1, x_f32, dy_f32, out_f32, mean != nullptr);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_sum_kernel, dim3(static_cast<uint32_t>((H + 63) / 64), db != nullptr ? 2 : 1), dim3(1024), 0,
                     stream, part, groups, static_cast<int>(H), dw, db);
  return hipGetLastError();
}

}  // namespace fp8q
