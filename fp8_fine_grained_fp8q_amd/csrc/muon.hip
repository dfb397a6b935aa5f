// Muon: the update of a weight matrix made orthogonal by Newton-Schulz products, for gfx950.
//
//   X = U / |U|_F;  `steps` times:  A = X X^T,  X = (a I + b A + c A^2) X,
// which takes every singular value s of X to s (a + b s^2 + c s^4) and leaves the singular vectors.
// U is a matrix, or the momentum M = beta M + g (Nesterov: g + beta M); then
//   p = p (1 - lr weight_decay) - lr scale X.
// X has the smaller of the two sizes, m, as its rows (n columns): tall matrices are worked on transposed.
//
// Three matrix products per step on the FP16 matrix instructions: A and C = a I + b A + c A^2, of which only the
// lower triangle of tiles is computed and mirrored, and C X (tall: X C).  5 steps of 4096 x 7168:
// 2 (m^2 n / 2 + m^3 / 2 + m^2 n) flops each = 2.1e12 in all.  X stays in the orientation of the matrix, once: the
// product that contracts over its columns reads it by rows, the other by columns (LDS's transposing reads).
//
// Numerics.  FP16 has 11 significant bits, three more than BF16, and its range is no matter with the usual coefficients:
// |X|_2 stays below 1.3 and operands are scaled by 2^12 (others: |X|_2 below 5.65, |C|_2 below 15.99).  Rounding X itself to 11 bits would drown the small singular
// values beside strong directions (a rank-1 matrix with a floor of noise: 1e-2 of the result's norm), as
// would rounding a + b A_ii + ..., where the terms cancel.  So X is kept in 15 bits, hi in FP16 and the rest lo in
// E4M3 (behind those the products' own 11 bits lose more, and FP16 would be another byte per element to read and
// write each step), the diagonal of A in FP32 apart from A, whose own is zero, and that of C in FP32 beside its rounded one.
// The products see hi and 11 bits of what is off the diagonal; lo and the diagonal's rest come in with FP32
// factors afterwards (muon_apply_kernel).  Result, off by, of its norm (a model of these roundings in 64 bits): smaller side
// 128 and more, 1e-4 to 9e-4 (normal, a few strong directions over noise, down to singular values of 1/500 of the norm),
// less than the rounding to BF16 (1.7e-3), and up to 6e-3 with a floor of 1/10000.  What is off the diagonals of A and C
// averages out over fewer elements below that: 64, 3e-3; 16, 2e-2; 8, 3e-2 at worst (one direction over a floor of 1/500;
// normal ones 1e-3, 2e-3 and 4e-3), against 1e-6 to 5e-5 with FP32 throughout.
//
// What bounds it.  Large: the matrix cores at the clock that the power limit leaves, and CUs that the last round of
// tiles leaves idle (C X of 4096 x 7168: 448 tiles on 256 CUs).  32 x 7168 x 2048 in 17.4 to 17.9 ms:
// C X 1.78 ms (1.08 PFLOP/s), of which the sums alone take 1.35 (1.41, what a large library product reaches) and
// lo, the factors and the stores the rest (its instance for wide matrices spills 20 bytes per thread); A 0.93, C 0.34,
// momentum and norm 0.95 (HBM), first X 0.79, which reads gradient and momentum again, the last C X with the parameters
// 2.41.  Reading lo after the products (1.89), storing hi without LDS (1.89), starting the CUs apart (no gain) and lo and
// hi by buffer addresses (1.80) did not help.  Small: the launches, each 4 to 9 us and none able to start before the one
// before it has ended.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "fp8q.h"
#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

namespace {

#define FP8Q_LDS __attribute__((address_space(3)))
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr float kScale = 4096.0f;  // of X, A and C as stored
constexpr int64_t kPad = 128;      // sizes of the stored matrices
constexpr int kThreads = 512;
constexpr int kPerSum = 8192;  // elements that a workgroup sums the squares of at a time
constexpr int64_t kSums = 16384;  // the most of these workgroups, for several matrices together

int64_t padded(int64_t v) { return (v + kPad - 1) / kPad * kPad; }

// ---------------------------------------------------------------------------------------
// Momentum, norm and the first X
// ---------------------------------------------------------------------------------------
struct Update {
  const void *grad;    // the matrix itself without momentum
  float *momentum;     // or null
  float beta, grad_scale;
  bool nesterov;
};

template <bool kF32>
__device__ __forceinline__ float value_at(const void *p, int64_t i) {
  return kF32 ? static_cast<const float *>(p)[i] : bf16_lo(static_cast<const uint16_t *>(p)[i]);
}

template <bool kF32>
__device__ __forceinline__ void load4(const void *p, int64_t i, float (&v)[4]) {
  if (kF32) {
    const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
    v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  }
}

// The update from a gradient and the new momentum.
__device__ __forceinline__ float update_of(const Update &u, float g, float m) {
  return u.nesterov ? __builtin_fmaf(u.beta, m, g * u.grad_scale) : m;
}

// Workgroup (x, y): kPerSum elements of matrix y, and every gridDim.x-th so many after them: the new momentum and
// the sum of the update's squares.
// In 64 bits, which hold the squares of every FP32 number.
template <bool kF32, bool kVector>
__global__ __launch_bounds__(256) void muon_momentum_kernel(const Update u, int64_t size, double *__restrict__ sums) {
  __shared__ double waves[4];
  double sum = 0.0;
  const int64_t end = (blockIdx.y + int64_t(1)) * size;
  int64_t first = blockIdx.y * size + static_cast<int64_t>(blockIdx.x) * kPerSum;
  for (; first < end; first += static_cast<int64_t>(gridDim.x) * kPerSum) {
#pragma unroll
    for (int k = 0; k < kPerSum / 2048; ++k) {
      const int64_t at = first + k * 2048 + threadIdx.x * 8;
      if (at >= end) break;
      const int n = end - at < 8 ? static_cast<int>(end - at) : 8;
      float g[8], m[8];
      if (kVector) {
        load8<kF32>(u.grad, at, g);
        if (u.momentum != nullptr) load8<true>(u.momentum, at, m);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          g[i] = i < n ? value_at<kF32>(u.grad, at + i) : 0.0f;
          m[i] = i < n && u.momentum != nullptr ? u.momentum[at + i] : 0.0f;
        }
      }
      if (u.momentum != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = __builtin_fmaf(u.beta, m[i], g[i] * u.grad_scale);
        if (kVector) {
          store8<true>(u.momentum, at, m);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < n) u.momentum[at + i] = m[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = u.momentum != nullptr ? update_of(u, g[i], m[i]) : g[i];
        sum += v * v;
      }
    }
  }
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    sums[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = (waves[0] + waves[1]) + (waves[2] + waves[3]);
}

// X as it is stored: hi in FP16, 11 bits, and lo in E4M3, 4 more, with hi + lo / kLow = kScale X, [Pp][Qp] in the
// orientation of the matrix itself, zeros in the padding.
struct Matrices {
  const _Float16 *hi;  // read
  _Float16 *next;      // written
  uint8_t *lo;         // both
  int64_t Pp, Qp;
};

constexpr float kLow = 256.0f;

// lo lies as a product's lanes take it: in 64 columns of a row, the four neighbours 16 j + 4 g .. + 3 at 16 g + 4 j, so
// that the 16 bytes at 16 g are those of one lane in four fragments.
__device__ __forceinline__ int64_t low_place(int64_t c) {
  return (c & ~int64_t(63)) + 16 * ((c >> 2) & 3) + 4 * ((c >> 4) & 3);
}

// Four values at lo's scale (kLow times hi's) as hi and lo.
__device__ __forceinline__ v4h split(v4f v, uint32_t &lo) {
  v4h hi;
  v4f rest;
#pragma unroll
  for (int k = 0; k < 4; ++k) hi[k] = static_cast<_Float16>(v[k] * (1.0f / kLow));
  // One rounding for both: the compiler may round a product or sum twice for one of two conversions and once
  // for the other, and where these differ lo would belong to another hi.
  asm volatile("" : "+v"(hi));
#pragma unroll
  for (int k = 0; k < 4; ++k) rest[k] = __builtin_fmaf(static_cast<float>(hi[k]), -kLow, v[k]);
  lo = pack4_e4m3(rest[0], rest[1], rest[2], rest[3]);
  return hi;
}

// lo at its scale.
__device__ __forceinline__ v4f low_of(uint32_t lo) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(lo), false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(lo), true);
  return v4f{a.x, a.y, b.x, b.y};
}

// Workgroup (x, y, z): 16 rows of 256 columns of matrix z, and every gridDim.y-th 16 after them.
template <bool kF32, bool kVector>
__global__ __launch_bounds__(256) void muon_start_kernel(const Update u, const double *__restrict__ sums, int count,
                                                         int64_t P, int64_t Q, const Matrices x) {
  __shared__ double waves[4];
  double sum = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < count; i += 256) sum += sums[static_cast<int64_t>(blockIdx.z) * count + i];
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = (waves[0] + waves[1]) + (waves[2] + waves[3]);
  // kLow kScale / |U| as a power of two, which may lie outside FP32, and a factor of 1/2 to 1: FP64 products cost twice
  // the time of the copy.
  int power = 0;
  const float factor = sum > 0.0 ? static_cast<float>(frexp(static_cast<double>(kLow * kScale) / sqrt(sum), &power)) : 0.0f;

  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + (threadIdx.x & 63) * 4;
  if (c >= x.Qp) return;
  // Pp is a multiple of 16: every wave takes four rows at once
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * 16 + (threadIdx.x >> 6) * 4; r0 < x.Pp; r0 += gridDim.y * 16) {
    float g[4][4], m[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = (blockIdx.z * P + r0 + i) * Q + c;
#pragma unroll
      for (int k = 0; k < 4; ++k) g[i][k] = m[i][k] = 0.0f;
      if (r0 + i >= P) continue;
      if (kVector) {  // Q % 4 == 0
        if (c < Q) {
          load4<kF32>(u.grad, at, g[i]);
          if (u.momentum != nullptr) load4<true>(u.momentum, at, m[i]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (c + k >= Q) break;
          g[i][k] = value_at<kF32>(u.grad, at + k);
          if (u.momentum != nullptr) m[i][k] = u.momentum[at + k];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v4f v;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = ldexpf(u.momentum != nullptr ? update_of(u, g[i][k], m[i][k]) : g[i][k], power) * factor;
      uint32_t lo;
      const v4h hi = split(v, lo);
      const int64_t to = (blockIdx.z * x.Pp + r0 + i) * x.Qp;
      *reinterpret_cast<v4h *>(x.next + to + c) = hi;
      *reinterpret_cast<uint32_t *>(x.lo + to + low_place(c)) = lo;
    }
  }
}

// ---------------------------------------------------------------------------------------
// Products, out = P Q with P's rows and Q's columns contiguous or not: an operand is "by rows" where the
// contracted index is contiguous, "by columns" where the output's is.  A workgroup of 8 waves
// (4 x 2) makes a tile of kTile x kTile; each wave kTile / 4 rows by kTile / 2 columns.
//
// Stages of 64 of the contracted index go to LDS by buffer_load ... lds in panels of 64 rows of 128 bytes (by
// rows: 64 of the output's rows; by columns: 64 of the contracted index by 64 columns); a wave moves 1 KB of
// every panel.  In a panel rows r and r + 8 of a group of 16 share a 256-byte line and the 16-byte
// chunks of a row are swapped among themselves, so that a fragment read touches every bank once: by rows
// ds_read_b128 takes one chunk of 16 rows (chunk ^ r mod 8), by columns ds_read_b64_tr_b16 two neighbouring
// chunks of 8 rows (chunk ^ 2 (r mod 4)) and turns them.
//
// The operand with the output's columns is the instruction's first one: a lane then owns one output row
// and four consecutive columns per fragment.
// ---------------------------------------------------------------------------------------
constexpr int kPanel = 8192;

__device__ __forceinline__ int panel_pos(int row, int slot) {
  return (row >> 4) * 2048 + (row & 7) * 256 + ((row >> 3) & 1) * 128 + slot * 16;
}

// One operand's part of a tile: where its panels come from.
template <bool kCols>
struct Source {
  const uint8_t *p;
  int64_t stride;  // bytes of a row
  int64_t bytes;   // by rows: of the tile's rows; by columns: of a stage
  int voff, stages;

  // By rows: rows [at, at + most) of `rows`; by columns: columns from `at` on, K rows.  Of the K / 64 stages all, or
  // `count` from `first` on.
  __device__ __forceinline__ Source(const _Float16 *from, int64_t at, int64_t rows, int most, int64_t ld, int64_t K,
                                    int first = 0, int count = 0) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    stride = ld * 2;
    stages = count > 0 ? count : static_cast<int>(K / 64);
    const int line = 4 * (wave & 1) + (lane >> 4), row = 16 * (wave >> 1) + line + 8 * ((lane >> 3) & 1);
    const int chunk = (lane & 7) ^ (kCols ? 2 * (line & 3) : line);
    voff = row * static_cast<int>(stride) + chunk * 16;
    if (kCols) {
      p = reinterpret_cast<const uint8_t *>(from + at);
      bytes = 64 * stride - at * 2;  // columns past the last are others' or zeros, and their output is not used
    } else {
      p = reinterpret_cast<const uint8_t *>(from + at * ld);
      bytes = (rows - at < most ? rows - at : most) * stride - first * 128;  // rows past the last are zeros
    }
    p += kCols ? first * 64 * stride : first * 128;
  }
  // The wave's 1 KB of panel i of stage s; past the last stage zeros without traffic, so that every wave
  // always has the same number of copies in flight.
  __device__ __forceinline__ void copy(int s, int i, uint8_t *panel) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint8_t *const from = kCols ? p + s * 64 * stride : p;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(from), static_cast<short>(0), s < stages ? static_cast<int>(bytes) : 0, 0x00020000);
    const int soff = kCols ? i * 128 : s * 128 + i * 64 * static_cast<int>(stride);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (FP8Q_LDS void *)(panel + wave * 1024), 16, voff, s < stages ? soff : 0, 0, 0);
  }
};

// A lane's places in LDS of the fragments first .. first + kCount - 1 (16 rows or columns each) of a region.
template <bool kCols, int kCount>
struct Places {
  uint32_t at[kCols ? kCount : 2];
  __device__ __forceinline__ explicit Places(int first) {
    const int l = threadIdx.x & 15, kg = (threadIdx.x & 63) >> 4;
    if (kCols) {
      const int k = 8 * kg + (l >> 2);
#pragma unroll
      for (int f = 0; f < kCount; ++f) {
        const int g = first + f, chunk = 2 * (g & 3) + ((l >> 1) & 1);
        at[f] = (g >> 2) * kPanel + panel_pos(k, chunk ^ (2 * (k & 3))) + 8 * (l & 1);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) at[h] = first * 2048 + panel_pos(l, (kg + 4 * h) ^ (l & 7));
    }
  }
  // x[h][f]: fragment first + f, contracted indices 32 h + 8 (lane / 16) + 0 .. 7, of the region at LDS address
  // `base`.  In assembly, with their wait: the compiler would wait for every copy in flight.
  template <int kN>
  __device__ __forceinline__ void read(v8h (&x)[2][kN], uint32_t base, int first) const {
    if constexpr (kCols) {
      v4s r[2][kN][2];
      if constexpr (kN == 1) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %4 offset:0\n\tds_read_b64_tr_b16 %1, %4 offset:1024\n\t"
            "ds_read_b64_tr_b16 %2, %4 offset:4096\n\tds_read_b64_tr_b16 %3, %4 offset:5120\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0][0]), "=&v"(r[0][0][1]), "=&v"(r[1][0][0]), "=&v"(r[1][0][1])
            : "v"(base + at[first + 0])
            : "memory");
      } else if constexpr (kN == 2) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8 offset:0\n\tds_read_b64_tr_b16 %1, %8 offset:1024\n\t"
            "ds_read_b64_tr_b16 %2, %9 offset:0\n\tds_read_b64_tr_b16 %3, %9 offset:1024\n\t"
            "ds_read_b64_tr_b16 %4, %8 offset:4096\n\tds_read_b64_tr_b16 %5, %8 offset:5120\n\t"
            "ds_read_b64_tr_b16 %6, %9 offset:4096\n\tds_read_b64_tr_b16 %7, %9 offset:5120\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0][0]), "=&v"(r[0][0][1]), "=&v"(r[0][1][0]), "=&v"(r[0][1][1]), "=&v"(r[1][0][0]),
              "=&v"(r[1][0][1]), "=&v"(r[1][1][0]), "=&v"(r[1][1][1])
            : "v"(base + at[first + 0]), "v"(base + at[first + 1])
            : "memory");
      } else if constexpr (kN == 3) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %12 offset:0\n\tds_read_b64_tr_b16 %1, %12 offset:1024\n\t"
            "ds_read_b64_tr_b16 %2, %13 offset:0\n\tds_read_b64_tr_b16 %3, %13 offset:1024\n\t"
            "ds_read_b64_tr_b16 %4, %14 offset:0\n\tds_read_b64_tr_b16 %5, %14 offset:1024\n\t"
            "ds_read_b64_tr_b16 %6, %12 offset:4096\n\tds_read_b64_tr_b16 %7, %12 offset:5120\n\t"
            "ds_read_b64_tr_b16 %8, %13 offset:4096\n\tds_read_b64_tr_b16 %9, %13 offset:5120\n\t"
            "ds_read_b64_tr_b16 %10, %14 offset:4096\n\tds_read_b64_tr_b16 %11, %14 offset:5120\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0][0]), "=&v"(r[0][0][1]), "=&v"(r[0][1][0]), "=&v"(r[0][1][1]), "=&v"(r[0][2][0]),
              "=&v"(r[0][2][1]), "=&v"(r[1][0][0]), "=&v"(r[1][0][1]), "=&v"(r[1][1][0]), "=&v"(r[1][1][1]),
              "=&v"(r[1][2][0]), "=&v"(r[1][2][1])
            : "v"(base + at[first + 0]), "v"(base + at[first + 1]), "v"(base + at[first + 2])
            : "memory");
      } else if constexpr (kN == 4) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %16 offset:0\n\tds_read_b64_tr_b16 %1, %16 offset:1024\n\t"
            "ds_read_b64_tr_b16 %2, %17 offset:0\n\tds_read_b64_tr_b16 %3, %17 offset:1024\n\t"
            "ds_read_b64_tr_b16 %4, %18 offset:0\n\tds_read_b64_tr_b16 %5, %18 offset:1024\n\t"
            "ds_read_b64_tr_b16 %6, %19 offset:0\n\tds_read_b64_tr_b16 %7, %19 offset:1024\n\t"
            "ds_read_b64_tr_b16 %8, %16 offset:4096\n\tds_read_b64_tr_b16 %9, %16 offset:5120\n\t"
            "ds_read_b64_tr_b16 %10, %17 offset:4096\n\tds_read_b64_tr_b16 %11, %17 offset:5120\n\t"
            "ds_read_b64_tr_b16 %12, %18 offset:4096\n\tds_read_b64_tr_b16 %13, %18 offset:5120\n\t"
            "ds_read_b64_tr_b16 %14, %19 offset:4096\n\tds_read_b64_tr_b16 %15, %19 offset:5120\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0][0]), "=&v"(r[0][0][1]), "=&v"(r[0][1][0]), "=&v"(r[0][1][1]), "=&v"(r[0][2][0]),
              "=&v"(r[0][2][1]), "=&v"(r[0][3][0]), "=&v"(r[0][3][1]), "=&v"(r[1][0][0]), "=&v"(r[1][0][1]),
              "=&v"(r[1][1][0]), "=&v"(r[1][1][1]), "=&v"(r[1][2][0]), "=&v"(r[1][2][1]), "=&v"(r[1][3][0]),
              "=&v"(r[1][3][1])
            : "v"(base + at[first + 0]), "v"(base + at[first + 1]), "v"(base + at[first + 2]),
              "v"(base + at[first + 3])
            : "memory");
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < kN; ++f)
          x[h][f] = __builtin_bit_cast(v8h, __builtin_shufflevector(r[h][f][0], r[h][f][1], 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      base += first * 2048;
      if constexpr (kN == 1) {
        asm volatile(
            "ds_read_b128 %0, %2 offset:0\n\tds_read_b128 %1, %3 offset:0\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(x[0][0]), "=&v"(x[1][0])
            : "v"(base + at[0]), "v"(base + at[1])
            : "memory");
      } else if constexpr (kN == 2) {
        asm volatile(
            "ds_read_b128 %0, %4 offset:0\n\tds_read_b128 %1, %4 offset:2048\n\t"
            "ds_read_b128 %2, %5 offset:0\n\tds_read_b128 %3, %5 offset:2048\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(x[0][0]), "=&v"(x[0][1]), "=&v"(x[1][0]), "=&v"(x[1][1])
            : "v"(base + at[0]), "v"(base + at[1])
            : "memory");
      } else if constexpr (kN == 3) {
        asm volatile(
            "ds_read_b128 %0, %6 offset:0\n\tds_read_b128 %1, %6 offset:2048\n\t"
            "ds_read_b128 %2, %6 offset:4096\n\tds_read_b128 %3, %7 offset:0\n\t"
            "ds_read_b128 %4, %7 offset:2048\n\tds_read_b128 %5, %7 offset:4096\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(x[0][0]), "=&v"(x[0][1]), "=&v"(x[0][2]), "=&v"(x[1][0]), "=&v"(x[1][1]), "=&v"(x[1][2])
            : "v"(base + at[0]), "v"(base + at[1])
            : "memory");
      } else if constexpr (kN == 4) {
        asm volatile(
            "ds_read_b128 %0, %8 offset:0\n\tds_read_b128 %1, %8 offset:2048\n\t"
            "ds_read_b128 %2, %8 offset:4096\n\tds_read_b128 %3, %8 offset:6144\n\t"
            "ds_read_b128 %4, %9 offset:0\n\tds_read_b128 %5, %9 offset:2048\n\t"
            "ds_read_b128 %6, %9 offset:4096\n\tds_read_b128 %7, %9 offset:6144\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(x[0][0]), "=&v"(x[0][1]), "=&v"(x[0][2]), "=&v"(x[0][3]), "=&v"(x[1][0]), "=&v"(x[1][1]),
              "=&v"(x[1][2]), "=&v"(x[1][3])
            : "v"(base + at[0]), "v"(base + at[1])
            : "memory");
      }
    }
  }
};

__device__ __forceinline__ uint32_t lds_address(const uint8_t *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const FP8Q_LDS uint8_t *)p));
}

template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Waits for the wave's LDS reads, then for the other waves.  Not __syncthreads(), whose fence would wait
// for the copies in flight.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// LDS that other lanes of the wave have written is read behind this.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ void in_order() { asm volatile("" ::: "memory"); }

template <int kTile>
struct Tile {
  static constexpr int kM = kTile / 64, kN = kTile / 32;  // fragments of a wave
  static constexpr int kLds = kTile == 192 ? 18 * kPanel : kTile == 64 ? 10 * kPanel : 16 * kPanel;
  v4f acc[kM][kN];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < kN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // acc += fragments a times fragments b of columns first .. first + kCount - 1
  template <int kCount>
  __device__ __forceinline__ void add(const v8h (&a)[2][kM], const v8h (&b)[2][kCount], int first) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < kCount; ++j)
#pragma unroll
        for (int i = 0; i < kM; ++i)
          acc[i][first + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[h][j], a[h][i], acc[i][first + j], 0, 0, 0);
  }
};

// Tiles of 256.  The two waves of a SIMD (w and w + 4) take turns: one multiplies while the other reads
// fragments from LDS and issues copies; a barrier ends each phase, and waves 0-3 run one phase ahead.  A
// stage is two of each: M0 reads the row fragments and the first half of the wave's columns (regions p
// and q0), C0 multiplies them, M1 reads the other half (region q1), C1 multiplies.  Regions are
// double buffered, 128 KB in all; a region is free two phases after its last read.  In M0 of stage
// s the copies of q1 of stage s + 1 are issued, in M1 those of p and q0 of stage s + 2, so that a
// copy has about one and a half stages (3000 cycles) to land.  Each wave waits at the end of its M phases
// for the copies that the phase after next reads, all but the eight issued last.
template <bool kPCols, bool kQCols>
__device__ __forceinline__ void multiply(Tile<256> &t, const Source<kPCols> &p, const Source<kQCols> &q, uint8_t *lds) {
  uint8_t *const p_0 = lds, *const p_1 = lds + 4 * kPanel, *const q0_0 = lds + 8 * kPanel, *const q0_1 = lds + 10 * kPanel,
                 *const q1_0 = lds + 12 * kPanel, *const q1_1 = lds + 14 * kPanel;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool lead = wave < 4;
  const Places<kPCols, 4> at_p((wave >> 1) * 4);
  const Places<kQCols, 4> at_q((wave & 1) * 4);
  auto copy_first = [&](int s, uint8_t *to_p, uint8_t *to_q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p.copy(s, i, to_p + i * kPanel);
#pragma unroll
    for (int i = 0; i < 2; ++i) q.copy(s, 2 * i, to_q + i * kPanel);
  };
  auto copy_second = [&](int s, uint8_t *to) {
#pragma unroll
    for (int i = 0; i < 2; ++i) q.copy(s, 2 * i + 1, to + i * kPanel);
  };
  t.clear();
  copy_first(0, p_0, q0_0);
  in_order();
  copy_second(0, q1_0);
  in_order();
  copy_first(1, p_1, q0_1);
  wait_copies<8>();
  meet();
  if (!lead) meet();
  v8h a[2][4], b[2][4];
  auto stage = [&](int s, uint8_t *sp, uint8_t *s0, uint8_t *s1, uint8_t *next1) {
    at_p.read(a, lds_address(sp), 0);
    at_q.read(b, lds_address(s0), 0);
    in_order();
    copy_second(s + 1, next1);
    wait_copies<8>();
    meet();
    t.add<4>(a, b, 0);
    meet();
    at_q.read(b, lds_address(s1), 0);
    in_order();
    copy_first(s + 2, sp, s0);
    wait_copies<8>();
    meet();
    t.add<4>(a, b, 4);
    meet();
  };
  for (int s = 0; s < p.stages; s += 2) {  // an even number
    stage(s, p_0, q0_0, q1_0, q1_1);
    stage(s + 1, p_1, q0_1, q1_1, q1_0);
  }
  if (lead) meet();
  wait_copies<0>();
}

// Tiles of 192: the same phases with three buffers for whole stages (144 KB).  In M0 of stage s all
// copies of stage s + 2 are issued, into the buffer that was last read two phases before.
template <bool kPCols, bool kQCols>
__device__ __forceinline__ void multiply(Tile<192> &t, const Source<kPCols> &p, const Source<kQCols> &q, uint8_t *lds) {
  uint8_t *const b_0 = lds, *const b_1 = lds + 6 * kPanel, *const b_2 = lds + 12 * kPanel;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool lead = wave < 4;
  const Places<kPCols, 3> at_p((wave >> 1) * 3);
  const Places<kQCols, 6> at_q((wave & 1) * 6);
  auto copy = [&](int s, uint8_t *to) {
#pragma unroll
    for (int i = 0; i < 3; ++i) p.copy(s, i, to + i * kPanel);
#pragma unroll
    for (int i = 0; i < 3; ++i) q.copy(s, i, to + (3 + i) * kPanel);
  };
  t.clear();
  copy(0, b_0);
  in_order();
  copy(1, b_1);
  wait_copies<6>();
  meet();
  if (!lead) meet();
  v8h a[2][3], b[2][3];
  auto stage = [&](int s, uint8_t *cur, uint8_t *free) {
    at_p.read(a, lds_address(cur), 0);
    at_q.read(b, lds_address(cur + 3 * kPanel), 0);
    in_order();
    copy(s + 2, free);
    meet();
    t.add<3>(a, b, 0);
    meet();
    at_q.read(b, lds_address(cur + 3 * kPanel), 3);
    wait_copies<6>();
    meet();
    t.add<3>(a, b, 3);
    meet();
  };
  for (int s = 0;;) {
    stage(s, b_0, b_2);
    if (++s == p.stages) break;
    stage(s, b_1, b_0);
    if (++s == p.stages) break;
    stage(s, b_2, b_1);
    if (++s == p.stages) break;
  }
  if (lead) meet();
  wait_copies<0>();
}

// Tiles of 128 and of 64, for few of them: what counts is the time until a stage arrives.  Four buffers for whole
// stages (128 KB) or five (80 KB, two workgroups per CU), every wave in step, all but one stage in flight.  With
// eight buffers and one workgroup tiles of 64 took 11.0 instead of 8.6 us (C X of 256 x 7168).
template <int kTile, bool kPCols, bool kQCols>
__device__ __forceinline__ void multiply_ring(Tile<kTile> &t, const Source<kPCols> &p, const Source<kQCols> &q, uint8_t *lds) {
  constexpr int kPanels = kTile / 64, kStage = 2 * kPanels * kPanel, kRing = Tile<kTile>::kLds / kStage;
  constexpr int kM = Tile<kTile>::kM, kN = Tile<kTile>::kN;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Places<kPCols, kM> at_p((wave >> 1) * kM);
  const Places<kQCols, kN> at_q((wave & 1) * kN);
  auto copy = [&](int s, uint8_t *to) {
#pragma unroll
    for (int i = 0; i < kPanels; ++i) p.copy(s, i, to + i * kPanel);
#pragma unroll
    for (int i = 0; i < kPanels; ++i) q.copy(s, i, to + (kPanels + i) * kPanel);
  };
  t.clear();
#pragma unroll
  for (int s = 0; s + 1 < kRing; ++s) {
    copy(s, lds + s * kStage);
    in_order();
  }
  int cur = 0, free = (kRing - 1) * kStage;
  for (int s = 0; s < p.stages; ++s) {
    wait_copies<(kRing - 2) * 2 * kPanels>();
    meet();  // the stage has landed, and every wave has read the one before it
    copy(s + kRing - 1, lds + free);
    v8h a[2][kM], b[2][kN];
    at_p.read(a, lds_address(lds) + cur, 0);
    at_q.read(b, lds_address(lds) + cur + kPanels * kPanel, 0);
    t.template add<kN>(a, b, 0);
    free = cur;
    cur = cur == (kRing - 1) * kStage ? 0 : cur + kStage;
  }
  wait_copies<0>();
}

template <bool kPCols, bool kQCols>
__device__ __forceinline__ void multiply(Tile<128> &t, const Source<kPCols> &p, const Source<kQCols> &q, uint8_t *lds) {
  multiply_ring(t, p, q, lds);
}
template <bool kPCols, bool kQCols>
__device__ __forceinline__ void multiply(Tile<64> &t, const Source<kPCols> &p, const Source<kQCols> &q, uint8_t *lds) {
  multiply_ring(t, p, q, lds);
}

// Memory from p on, beyond whose end loads give zeros and stores write nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), static_cast<short>(0), static_cast<int>(bytes), 0x00020000);
}

// The lane's first row and column in the tile; fragment (i, j) is 16 i rows and 16 j columns further.
template <int kTile>
__device__ __forceinline__ void lane_place(int &row, int &col) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  row = (wave >> 1) * (kTile / 4) + (lane & 15);
  col = (wave & 1) * (kTile / 2) + (lane >> 4) * 4;
}

// Writes a wave's kTile / 4 x kTile / 2 block of FP16 values (v: its fragments) to out[row][column] and, if `mirror`, to
// out[column][row], 16 bytes per lane: through LDS, 16 bytes behind each row so that 16 of them use all
// banks.  r0, c0: the tile's place in out, whose sizes are multiples of 8.
template <int kTile>
__device__ __forceinline__ void store_block(const v4h (&v)[Tile<kTile>::kM][Tile<kTile>::kN], uint8_t *lds, _Float16 *out,
                                            int64_t r0, int64_t c0, int64_t rows_end, int64_t cols_end, int64_t ld,
                                            bool mirror) {
  constexpr int kM = Tile<kTile>::kM, kN = Tile<kTile>::kN, kHalf = (kM + 1) / 2;  // at most two parts of 32 rows
  constexpr int kRow = kN * 32 + 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 15, kg = lane >> 4;
  uint8_t *const mine = lds + wave * (kHalf * 16 * kRow);
  static_assert(8 * kHalf * 16 * kRow <= Tile<kTile>::kLds, "the blocks fit");
  r0 += (wave >> 1) * (kTile / 4);
  c0 += (wave & 1) * (kTile / 2);
#pragma unroll
  for (int part = 0; part < kM; part += kHalf) {
    constexpr int kChunks = kN * 2;  // of 16 bytes in a row
    const int rows = (kM - part < kHalf ? kM - part : kHalf) * 16;
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
      if (part + i < kM)
#pragma unroll
        for (int j = 0; j < kN; ++j)
          *reinterpret_cast<v4h *>(mine + (16 * i + l) * kRow + (16 * j + 4 * kg) * 2) = v[part + i][j];
    wave_order();
    for (int n = lane; n < rows * kChunks; n += 64) {
      const int r = n / kChunks, c = n % kChunks * 8;
      const int64_t i = r0 + part * 16 + r, j = c0 + c;
      if (i < rows_end && j < cols_end)
        *reinterpret_cast<uint4 *>(out + i * ld + j) = *reinterpret_cast<const uint4 *>(mine + r * kRow + c * 2);
    }
    if (mirror) {
      // 16 columns by 8 rows for each 16 lanes: lane l gets column l
      const int blocks = rows / 8;
      for (int n = kg; n < blocks * kN; n += 4) {
        const int rb = n % blocks, cb = n / blocks;
        const uint8_t *const at = mine + (8 * rb + (l >> 2)) * kRow + (16 * cb + 4 * (l & 3)) * 2;
        const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FP8Q_LDS v4s *)at);
        const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FP8Q_LDS v4s *)(at + 4 * kRow));
        const int64_t i = r0 + part * 16 + 8 * rb, j = c0 + 16 * cb + l;
        if (i < rows_end && j < cols_end)
          *reinterpret_cast<uint4 *>(out + j * ld + i) =
              __builtin_bit_cast(uint4, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
    wave_order();
  }
}

// Unit of a workgroup: each XCD (blockIdx % 8) takes a run of neighbouring tiles, which share operands in
// its L2.
__device__ __forceinline__ int64_t unit_of(int64_t units) {
  const int64_t per = (units + 7) / 8;
  return (blockIdx.x & 7) * per + (blockIdx.x >> 3);
}

// The u-th pair i >= j.
__device__ __forceinline__ void triangle(int u, int &i, int &j) {
  i = static_cast<int>((sqrtf(8.0f * static_cast<float>(u) + 1.0f) - 1.0f) * 0.5f);
  while (i * (i + 1) / 2 > u) --i;
  while ((i + 1) * (i + 2) / 2 <= u) ++i;
  j = u - i * (i + 1) / 2;
}

struct Coefficients {
  float a, b, c;
};

// kSquare false: A = X X^T (or X^T X, kCols), its own diagonal zero, and the diagonal in FP32.  true: C = a I + b A +
// c A^2 from these, its diagonal rounded to FP16 like the rest, and for each row the diagonal d in FP32
// and its quotient by the rounded one, {d, d / rounded}.  m: the size of A.
template <int kTile, bool kSquare, bool kCols>
__global__ __launch_bounds__(kThreads, 2) void muon_symmetric_kernel(const _Float16 *__restrict__ from, int64_t ld,
                                                                     int64_t K, int64_t m, int G,
                                                                     const float *__restrict__ diagonal_in,
                                                                     Coefficients co, _Float16 *__restrict__ out,
                                                                     float *__restrict__ diagonal,
                                                                     float2 *__restrict__ pairs, int splits,
                                                                     float *__restrict__ parts) {
  const int tiles = static_cast<int>((m + kTile - 1) / kTile), per = tiles * (tiles + 1) / 2;
  const int64_t all = static_cast<int64_t>(per) * G * splits;
  int64_t unit = unit_of(all);
  if (unit >= all) return;
  const int part = static_cast<int>(unit % splits);
  unit /= splits;
  const int g = static_cast<int>(unit / per);
  int ti, tj;
  triangle(static_cast<int>(unit % per), ti, tj);
  const int64_t r0 = static_cast<int64_t>(ti) * kTile, c0 = static_cast<int64_t>(tj) * kTile;
  const _Float16 *x = from + g * m * K;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tile<kTile>::kLds];
  constexpr int kM = Tile<kTile>::kM, kN = Tile<kTile>::kN;
  const float *const d_in = kSquare ? diagonal_in + g * m : nullptr;
  int row, col;
  lane_place<kTile>(row, col);
  v4h h[kM][kN];
  v4f dj[kSquare ? kN : 1];
  auto read_own = [&]() {  // A's own tile, all of it on its way at once
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int64_t c = c0 + col + 16 * j;
      dj[j] = c < m ? *reinterpret_cast<const v4f *>(d_in + c) : v4f{};
    }
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int64_t r = r0 + row + 16 * i, c = c0 + col + 16 * j;
        h[i][j] = r < m && c < m ? *reinterpret_cast<const v4h *>(x + r * m + c) : v4h{};
      }
  };
  // before the products where there are registers for it
  if constexpr (kSquare && kTile != 256) read_own();
  in_order();
  Tile<kTile> t;
  if constexpr (kTile == 64 && !kSquare) {
    const int stages = static_cast<int>(K / 64), first = stages * part / splits;
    const int count = stages * (part + 1) / splits - first;
    multiply(t, Source<kCols>(x, r0, m, kTile, ld, K, first, count), Source<kCols>(x, c0, m, kTile, ld, K, first, count),
             lds);
    if (splits > 1) {  // muon_sum_kernel adds the parts up
      float *const to = parts + (unit * splits + part) * (kTile * kTile) + row * kTile + col;
#pragma unroll
      for (int i = 0; i < Tile<kTile>::kM; ++i)
#pragma unroll
        for (int j = 0; j < Tile<kTile>::kN; ++j) *reinterpret_cast<v4f *>(to + i * 16 * kTile + j * 16) = t.acc[i][j];
      return;
    }
  } else {
    multiply(t, Source<kCols>(x, r0, m, kTile, ld, K), Source<kCols>(x, c0, m, kTile, ld, K), lds);
  }
  if constexpr (kSquare && kTile == 256) read_own();
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    const int64_t r = r0 + row + 16 * i;
    const float di = kSquare && r < m ? d_in[r] : 0.0f;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int64_t c = c0 + col + 16 * j;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float s = t.acc[i][j][k] * (1.0f / kScale);
        if (r == c + k) {
          s *= 1.0f / kScale;
          if constexpr (kSquare) {
            const float d = __builtin_fmaf(co.c, __builtin_fmaf(di, di, s), __builtin_fmaf(co.b, di, co.a));
            s = d * kScale;
            const float rounded = static_cast<float>(static_cast<_Float16>(s));  // s is exact, and rounded alike below
            // below 2^-13 FP16 has fewer bits, and what they lose is nothing beside the other rows
            if (r < m) pairs[g * m + r] = make_float2(d, fabsf(rounded) >= 0x1p-13f ? s / rounded : 1.0f);
          } else {
            if (r < m) diagonal[g * m + r] = s;
            s = 0.0f;
          }
        } else if constexpr (kSquare) {
          const float e = static_cast<float>(h[i][j][k]);
          s = __builtin_fmaf(co.c, __builtin_fmaf(di + dj[j][k], e, s), co.b * e);
        }
        h[i][j][k] = static_cast<_Float16>(s);
      }
    }
  }
  meet();  // every wave's copies are done, and its reads
  store_block<kTile>(h, lds, out + g * m * m, r0, c0, m, m, m, ti != tj);
}

// A and its diagonal from the parts of its tiles of 64: workgroup (x, y) takes 16 rows of tile y of all.
__global__ __launch_bounds__(256) void muon_sum_kernel(const float *__restrict__ parts, int splits, int64_t m, int tiles,
                                                       _Float16 *__restrict__ out, float *__restrict__ diagonal) {
  const int per = tiles * (tiles + 1) / 2, g = blockIdx.y / per;
  int ti, tj;
  triangle(blockIdx.y % per, ti, tj);
  const int row = blockIdx.x * 16 + (threadIdx.x >> 4), col = (threadIdx.x & 15) * 4;
  const float *from = parts + static_cast<int64_t>(blockIdx.y) * splits * (64 * 64) + row * 64 + col;
  v4f sum = {};
#pragma unroll 8
  for (int s = 0; s < splits; ++s) sum += *reinterpret_cast<const v4f *>(from + s * (64 * 64));
  const int64_t i = ti * 64 + row, j = tj * 64 + col;
  _Float16 *const o = out + g * m * m;
  v4h h;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float v = sum[k] * (1.0f / kScale);
    if (i == j + k) {
      diagonal[g * m + i] = v * (1.0f / kScale);
      v = 0.0f;
    }
    h[k] = static_cast<_Float16>(v);
    if (ti != tj) o[(j + k) * m + i] = h[k];
  }
  *reinterpret_cast<v4h *>(o + i * m + j) = h;
}

struct Result {
  uint16_t *out;    // BF16 [G][P][Q], or null
  float *param;     // FP32 [G][P][Q]
  uint16_t *copy;   // BF16, the new param, or null
  const float *lr;  // device, or null
  float lr_host, decay, scale;
  int64_t P, Q;
};

// The parameters at row i, columns j .. j + 3 of matrix g, if there is a step to take and they are aligned.
__device__ __forceinline__ v4f old_param(const Result &res, int64_t g, int64_t i, int64_t j) {
  if (res.param == nullptr || (res.Q & 3) != 0 || i >= res.P || j >= res.Q) return v4f{};
  return *reinterpret_cast<const v4f *>(res.param + (g * res.P + i) * res.Q + j);
}

// The result there, from kLow kScale X and old_param's.
__device__ __forceinline__ void finish(const Result &res, int64_t g, int64_t i, int64_t j, v4f v, v4f p, float keep,
                                       float step) {
  if (i >= res.P) return;
  const int64_t at = (g * res.P + i) * res.Q + j;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] *= 1.0f / (kLow * kScale);
  if ((res.Q & 3) == 0) {
    if (j >= res.Q) return;
    if (res.param == nullptr) {
      *reinterpret_cast<uint2 *>(res.out + at) = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = p[k] * keep - step * v[k];
    *reinterpret_cast<v4f *>(res.param + at) = p;
    if (res.copy != nullptr)
      *reinterpret_cast<uint2 *>(res.copy + at) = make_uint2(pack2_bf16(p[0], p[1]), pack2_bf16(p[2], p[3]));
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (j + k >= res.Q) break;
    if (res.param == nullptr) {
      res.out[at + k] = static_cast<uint16_t>(pack2_bf16(v[k], 0.0f));
    } else {
      const float one = res.param[at + k] * keep - step * v[k];
      res.param[at + k] = one;
      if (res.copy != nullptr) res.copy[at + k] = static_cast<uint16_t>(pack2_bf16(one, 0.0f));
    }
  }
}

// finish for a tile whose columns all lie inside the aligned parameters: rows past the last are beyond the buffers'
// ends, and an address is a register (with 64-bit addresses and a branch for each fragment the last product of
// 32 x 7168 x 2048 took 2.74 instead of 2.40 ms).  Two rows of fragments at a time were no faster.
template <int kTile>
__device__ __forceinline__ void step_rows(const Result &res, int64_t g, int64_t r0, int64_t c0, const Tile<kTile> &t,
                                          float keep, float step) {
  constexpr int kM = Tile<kTile>::kM, kN = Tile<kTile>::kN;
  if (r0 >= res.P) return;
  const int64_t first = (g * res.P + r0) * res.Q + c0, rows = res.P - r0 < kTile ? res.P - r0 : kTile;
  const int size = static_cast<int>((rows * res.Q - c0) * 4), line = static_cast<int>(res.Q) * 4;
  const __amdgpu_buffer_rsrc_t param = buffer(res.param + first, size);
  const __amdgpu_buffer_rsrc_t copy = buffer(res.copy + first, res.copy != nullptr ? size / 2 : 0);
  int row, col;
  lane_place<kTile>(row, col);
  const int at = row * line + col * 4;
  step *= 1.0f / (kLow * kScale);
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    const int to = at + i * 16 * line;
    v4i old[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) old[j] = __builtin_amdgcn_raw_buffer_load_b128(param, to, j * 64, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      v4f v = __builtin_bit_cast(v4f, old[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = v[k] * keep - step * t.acc[i][j][k];
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, v), param, to, j * 64, 0);
      const v2i half = {static_cast<int>(pack2_bf16(v[0], v[1])), static_cast<int>(pack2_bf16(v[2], v[3]))};
      if (res.copy != nullptr) __builtin_amdgcn_raw_buffer_store_b64(half, copy, to >> 1, j * 32, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Tiles of C X.  Raster: 8 tiles of rows at a time, so that an XCD's run reads few panels.
__device__ __forceinline__ void raster(int u, int rows, int cols, int &i, int &j) {
  const int band = 8 * cols, first = u / band * 8;
  const int height = rows - first < 8 ? rows - first : 8;
  const int in = u % band;
  i = first + in % height;
  j = in / height;
}

// X = C X (kTall: the transposed matrix X = X C) from the products with hi; kLast: the result, [P][Q], in its place.
// With C's diagonal d rounded to dh in the product, row i (tall: column j) of it is multiplied by d / dh, which
// makes dh hi exact and is within the rounding of what is off the diagonal, and d lo is added: hi is not
// read again.
template <int kTile, bool kLast, bool kTall>
__global__ __launch_bounds__(kThreads, 2) void muon_apply_kernel(const _Float16 *__restrict__ c,
                                                                 const float2 *__restrict__ pairs, const Matrices x,
                                                                 int G, const Result res) {
  const int64_t Pp = x.Pp, Qp = x.Qp, m = kTall ? Qp : Pp;
  const int rows = static_cast<int>((Pp + kTile - 1) / kTile), cols = static_cast<int>((Qp + kTile - 1) / kTile);
  const int64_t per = static_cast<int64_t>(rows) * cols, unit = unit_of(per * G);
  if (unit >= per * G) return;
  const int64_t g = unit / per;
  int ti, tj;
  raster(static_cast<int>(unit % per), rows, cols, ti, tj);
  const int64_t r0 = static_cast<int64_t>(ti) * kTile, c0 = static_cast<int64_t>(tj) * kTile;
  const _Float16 *const hi = x.hi + g * Pp * Qp, *const cg = c + g * m * m;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tile<kTile>::kLds];
  constexpr int kM = Tile<kTile>::kM, kN = Tile<kTile>::kN;
  Tile<kTile> t;
  uint8_t *const lo = x.lo + g * Pp * Qp;
  _Float16 *const next = x.next + g * Pp * Qp;
  const float2 *const d = pairs + g * m;
  int row, col;
  lane_place<kTile>(row, col);
  // The lane's part of lo: kWide fragments of a row at a time.  Read before the products, which hide it.
  constexpr int kWide = kN % 4 == 0 ? 4 : 2;
  typedef uint32_t Low __attribute__((ext_vector_type(kWide)));
  auto low_at = [&](int i, int j) {
    return reinterpret_cast<Low *>(lo + (r0 + row + 16 * i) * Qp + low_place(c0 + col + 16 * j));
  };
  auto inside = [&](int i, int j) { return r0 + row + 16 * i < Pp && c0 + col + 16 * j < Qp; };
  Low low[kM][kN / kWide];
#pragma unroll
  for (int i = 0; i < kM; ++i)
#pragma unroll
    for (int j = 0; j < kN; j += kWide) low[i][j / kWide] = inside(i, j) ? *low_at(i, j) : Low{};
  in_order();
  if constexpr (kTall)
    multiply(t, Source<false>(hi, r0, Pp, kTile, Qp, m), Source<false>(cg, c0, m, kTile, m, m), lds);
  else
    multiply(t, Source<false>(cg, r0, m, kTile, m, m), Source<true>(hi, c0, Qp, kTile, Qp, m), lds);
  const float lr = kLast && res.param != nullptr ? (res.lr != nullptr ? *res.lr : res.lr_host) : 0.0f;
  const float keep = 1.0f - lr * res.decay, step = lr * res.scale;
  float2 d_row[kM];
  if constexpr (!kTall)
#pragma unroll
    for (int i = 0; i < kM; ++i) d_row[i] = r0 + row + 16 * i < Pp ? d[r0 + row + 16 * i] : make_float2(0.0f, 0.0f);
  __builtin_amdgcn_sched_barrier(0);
  v4h h[kLast ? 1 : kM][kLast ? 1 : kN];
  if constexpr (kTall) {  // columns' factors, four at a time for all rows
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int64_t c = c0 + col + 16 * j;
      v4f d01 = {}, d23 = {};
      if (c < Qp) {
        d01 = *reinterpret_cast<const v4f *>(d + c);
        d23 = *reinterpret_cast<const v4f *>(d + c + 2);
      }
      const v4f by = {d01[0], d01[2], d23[0], d23[2]}, turn = {d01[1], d01[3], d23[1], d23[3]};
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        const v4f rest = low_of(low[i][j / kWide][j % kWide]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          t.acc[i][j][k] = __builtin_fmaf(by[k], rest[k], t.acc[i][j][k] * (turn[k] * (kLow / kScale)));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const v4f rest = low_of(low[i][j / kWide][j % kWide]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          t.acc[i][j][k] = __builtin_fmaf(d_row[i].x, rest[k], t.acc[i][j][k] * (d_row[i].y * (kLow / kScale)));
      }
  }
  if constexpr (kLast) {
    if (res.param != nullptr && (res.Q & 3) == 0 && c0 + kTile <= res.Q) {
      step_rows<kTile>(res, g, r0, c0, t, keep, step);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    if constexpr (kLast) {
      v4f p[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) p[j] = old_param(res, g, r0 + row + 16 * i, c0 + col + 16 * j);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (inside(i, j)) finish(res, g, r0 + row + 16 * i, c0 + col + 16 * j, t.acc[i][j], p[j], keep, step);
    } else {
#pragma unroll
      for (int j = 0; j < kN; j += kWide) {
        Low rest;
#pragma unroll
        for (int k = 0; k < kWide; ++k) {
          uint32_t one;
          h[i][j + k] = split(t.acc[i][j + k], one);
          rest[k] = one;
        }
        if (inside(i, j)) *low_at(i, j) = rest;
      }
    }
  }
  if constexpr (!kLast) {
    meet();  // every wave's copies are done, and its reads
    store_block<kTile>(h, lds, next, r0, c0, Pp, Qp, Qp, false);
  }
}

// The workspace: sums of squares, X (hi twice, lo), A, C and their diagonals.
constexpr int64_t kFewTiles = 256;  // tiles of 64 and their parts, one for each CU

struct Layout {
  int64_t G, P, Q, Pp, Qp, m, count;  // count: workgroups that sum a matrix's squares
  int64_t tiles, splits;              // of a matrix's A in tiles of 64, and parts of each
  int64_t sums, hi[2], lo, a, c, da, dc, parts, bytes;
  Layout(int64_t G, int64_t P, int64_t Q) : G(G), P(P), Q(Q) {
    Pp = padded(P);
    Qp = padded(Q);
    m = Pp < Qp ? Pp : Qp;
    count = (P * Q + kPerSum - 1) / kPerSum;
    const int64_t most = G < kSums ? kSums / G : 1;
    count = count < most ? count : most;
    int64_t at = 0;
    auto take = [&](int64_t size) {
      const int64_t here = at;
      at += (size + 255) / 256 * 256;
      return here;
    };
    sums = take(8 * G * count);
    hi[0] = take(2 * G * Pp * Qp);
    hi[1] = take(2 * G * Pp * Qp);
    lo = take(G * Pp * Qp);
    a = take(2 * G * m * m);
    c = take(2 * G * m * m);
    da = take(4 * G * m);
    dc = take(8 * G * m);
    // A long sum of few tiles is split, at least 4 stages each.  Whole calls: 256 x 7168 (10 tiles, 112 stages) 122 us (in
    // tiles of 128 144), 896 x 7168 (105 tiles in 2 parts) 276 (in one 308); two parts for each CU 384 x 7168 143 -> 147.
    // Sums of less than 32 stages are over before muon_sum_kernel's launch would pay.
    tiles = (m / 64) * (m / 64 + 1) / 2;
    const int64_t stages = (Pp < Qp ? Qp : Pp) / 64, room = kFewTiles / (tiles * G);
    splits = stages / 4 < room ? stages / 4 : room;
    splits = stages < 32 || splits < 2 ? 1 : (splits > 16 ? 16 : splits);
    parts = take(splits > 1 ? 4 * 64 * 64 * G * tiles * splits : 0);
    bytes = at;
  }
};

// The tile size with the least time, by rounds over the CUs: smaller tiles fill them better and need more of the
// operands' bytes per product.  Whole calls (5 steps), in us, with all products in tiles of one size and by this rule:
//                  256    192    128     64   rule
//   300 x 1000     349    288    162     98     98
//   1400 x 1400    569    465    266    181    181
//   2000 x 2000    736    583    354    434    358
//   16 x 512 x 512 367    296    176    199    175
//   2304 x 5000   1035   1037    804   1017    673
//   4096 x 7168   2206   2495   3086   4161   2148
// (A of the last: 253 tiles of 192 in 132 us, 136 of 256 in 156.)
template <class Units>
int tile_for(Units units, int64_t cus) {
  int best = 256;
  double least = 0;
  for (int tile : {256, 192, 128, 64}) {
    const double rounds = static_cast<double>((units(tile) + cus - 1) / cus);
    const double time = rounds * tile * tile * (tile == 256 ? 1.0 : tile == 192 ? 1.1 : tile == 128 ? 1.4 : 2.5);
    if (least == 0 || time < least) {
      least = time;
      best = tile;
    }
  }
  return best;
}

template <class F>
void with_tile(int tile, F f) {
  if (tile == 256)
    f(std::integral_constant<int, 256>{});
  else if (tile == 192)
    f(std::integral_constant<int, 192>{});
  else if (tile == 128)
    f(std::integral_constant<int, 128>{});
  else
    f(std::integral_constant<int, 64>{});
}

hipError_t run(const Layout &w, const Update &u, bool f32, const Coefficients &co, int64_t steps, const Result &res,
               void *workspace, hipStream_t stream) {
  uint8_t *const ws = static_cast<uint8_t *>(workspace);
  auto halves = [&](int64_t at) { return reinterpret_cast<_Float16 *>(ws + at); };
  auto floats = [&](int64_t at) { return reinterpret_cast<float *>(ws + at); };
  double *const sums = reinterpret_cast<double *>(ws + w.sums);
  const bool tall = w.P > w.Q;
  const int64_t cus = device_cu_count();
  const int G = static_cast<int>(w.G);
  Matrices x = {nullptr, halves(w.hi[0]), ws + w.lo, w.Pp, w.Qp};
  {
    const bool vector = w.P * w.Q % 8 == 0;
    const dim3 grid(static_cast<uint32_t>(w.count), static_cast<uint32_t>(G)), block(256);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, u, w.P * w.Q, sums); };
    if (f32)
      vector ? go(muon_momentum_kernel<true, true>) : go(muon_momentum_kernel<true, false>);
    else
      vector ? go(muon_momentum_kernel<false, true>) : go(muon_momentum_kernel<false, false>);
    // Every workgroup adds up the sums first: of many, a thread takes 16 rows instead of 4.
    const int64_t columns = (w.Qp + 255) / 256;
    int64_t bands = w.Pp / 16;
    if (columns * bands * w.G > 16 * cus) bands = (bands + 3) / 4;
    const dim3 tiles(static_cast<uint32_t>(columns), static_cast<uint32_t>(bands < 65535 ? bands : 65535),
                     static_cast<uint32_t>(G));
    auto start = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, tiles, block, 0, stream, u, sums, static_cast<int>(w.count), w.P, w.Q, x);
    };
    if (f32)
      w.Q % 4 == 0 ? start(muon_start_kernel<true, true>) : start(muon_start_kernel<true, false>);
    else
      w.Q % 4 == 0 ? start(muon_start_kernel<false, true>) : start(muon_start_kernel<false, false>);
  }
  auto tiles = [](int64_t size, int tile) { return (size + tile - 1) / tile; };
  auto triangle_units = [&](int tile) { return w.G * tiles(w.m, tile) * (tiles(w.m, tile) + 1) / 2; };
  auto apply_units = [&](int tile) { return w.G * tiles(w.Pp, tile) * tiles(w.Qp, tile); };
  const int square = tile_for(triangle_units, cus), sym = w.splits > 1 ? 64 : square, app = tile_for(apply_units, cus);
  auto grid_of = [](int64_t units) { return dim3(static_cast<uint32_t>((units + 7) / 8 * 8)); };
  for (int64_t s = 0; s < steps; ++s) {
    x.hi = halves(w.hi[s & 1]);
    x.next = halves(w.hi[(s + 1) & 1]);
    auto symmetric = [&](auto kernel, int tile, const _Float16 *from, int64_t ld, int64_t K, const float *d_in, _Float16 *to,
                         int64_t splits) {
      hipLaunchKernelGGL(kernel, grid_of(triangle_units(tile) * splits), dim3(kThreads), 0, stream, from, ld, K, w.m, G, d_in,
                         co, to, floats(w.da), reinterpret_cast<float2 *>(ws + w.dc), static_cast<int>(splits),
                         floats(w.parts));
    };
    with_tile(sym, [&](auto tile) {
      constexpr int kT = decltype(tile)::value;
      if (tall)
        symmetric(muon_symmetric_kernel<kT, false, true>, kT, x.hi, w.Qp, w.Pp, nullptr, halves(w.a), w.splits);
      else
        symmetric(muon_symmetric_kernel<kT, false, false>, kT, x.hi, w.Qp, w.Qp, nullptr, halves(w.a), w.splits);
    });
    if (w.splits > 1)
      hipLaunchKernelGGL(muon_sum_kernel, dim3(4, static_cast<uint32_t>(w.G * w.tiles)), dim3(256), 0, stream,
                         floats(w.parts), static_cast<int>(w.splits), w.m, static_cast<int>(w.m / 64), halves(w.a),
                         floats(w.da));
    with_tile(square, [&](auto tile) {
      constexpr int kT = decltype(tile)::value;
      symmetric(muon_symmetric_kernel<kT, true, false>, kT, halves(w.a), w.m, w.m, floats(w.da), halves(w.c), 1);
    });
    with_tile(app, [&](auto tile) {
      constexpr int kT = decltype(tile)::value;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_of(apply_units(kT)), dim3(kThreads), 0, stream, halves(w.c),
                           reinterpret_cast<const float2 *>(ws + w.dc), x, G, res);
      };
      if (s + 1 < steps)
        tall ? go(muon_apply_kernel<kT, false, true>) : go(muon_apply_kernel<kT, false, false>);
      else
        tall ? go(muon_apply_kernel<kT, true, true>) : go(muon_apply_kernel<kT, true, false>);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

int64_t muon_workspace(int64_t G, int64_t P, int64_t Q) { return Layout(G, P, Q).bytes; }

bool muon_grids_fit(int64_t G, int64_t P, int64_t Q) {
  const Layout w(G, P, Q);
  const int64_t units = (w.Pp / 64) * (w.Qp / 64);  // the smallest tiles, of which a triangle has fewer
  return G <= 65535 && grid_fits(w.count, 256) && units < (int64_t(1) << 31) / kThreads &&
         grid_fits(G * units + 8, kThreads);
}

hipError_t launch_orthogonalize(const void *x, bool f32, int64_t G, int64_t P, int64_t Q, const fp8q_newton_schulz &ns,
                                uint16_t *out, void *workspace, hipStream_t stream) {
  const Update u = {x, nullptr, 0.0f, 1.0f, false};
  const Coefficients co = {static_cast<float>(ns.a), static_cast<float>(ns.b), static_cast<float>(ns.c)};
  const Result res = {out, nullptr, nullptr, nullptr, 0.0f, 0.0f, 0.0f, P, Q};
  return run(Layout(G, P, Q), u, f32, co, ns.steps, res, workspace, stream);
}

hipError_t launch_muon(float *param, const void *grad, bool f32, float *momentum, int64_t G, int64_t P, int64_t Q,
                       const fp8q_muon_hyper &h, uint16_t *copy, void *workspace, hipStream_t stream) {
  const Update u = {grad, momentum, static_cast<float>(h.beta), static_cast<float>(h.grad_scale), h.nesterov != 0};
  const Coefficients co = {static_cast<float>(h.ns.a), static_cast<float>(h.ns.b), static_cast<float>(h.ns.c)};
  const Result res = {nullptr, param, copy, h.device_lr, static_cast<float>(h.lr), static_cast<float>(h.weight_decay),
                      static_cast<float>(h.scale), P, Q};
  return run(Layout(G, P, Q), u, f32, co, h.ns.steps, res, workspace, stream);
}

}  // namespace fp8q
