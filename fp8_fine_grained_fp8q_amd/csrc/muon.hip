// Muon: the update of a weight matrix made orthogonal by Newton-Schulz products, for gfx950.
//
//   X = U / |U|_F;  `steps` times:  A = X X^T,  X = (a I + b A + c A^2) X,
// which takes every singular value s of X to s (a + b s^2 + c s^4) and leaves the singular vectors.
// U is a matrix, or the momentum M = beta M + g (Nesterov: g + beta M); then
//   p = p (1 - lr weight_decay) - lr scale X.
// X has the smaller of the two sizes, m, as its rows (n columns): tall matrices are worked on transposed.
//
// Three matrix products per step, all as P Q^T of operands with contiguous rows, on the FP16 matrix
// instructions: A (lower triangle of tiles, mirrored), C = a I + b A + c A^2 (likewise), C X with X^T kept
// beside X.  5 steps of 4096 x 7168: 2 (m^2 n / 2 + m^3 / 2 + m^2 n) flops each = 2.1e12 in all.
//
// Numerics.  FP16 has 11 significant bits, three more than BF16, and its range is no matter: |X|_2 stays
// below 1.3 and operands are scaled by 2^12.  Rounding X itself to 11 bits would drown the small singular
// values beside strong directions (a rank-1 matrix with a floor of noise: 1e-2 of the result's norm), as
// would rounding a + b A_ii + ..., where the terms cancel.  So X is kept in 22 bits, as two FP16 numbers;
// the diagonals of A and C are kept in FP32 apart from the matrices, whose diagonals are zero; and the
// diagonal's part of C X is formed from the 22 bits in FP32.  Products see 11 bits of what is off
// the diagonal.  Result: 1e-4 to 9e-4 of its norm off (normal, rank-1 and rank-16 matrices with noise),
// less than the rounding to BF16 (1.7e-3).
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
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));

constexpr float kScale = 4096.0f;  // of X, A and C as stored
constexpr int64_t kPad = 128;      // sizes of the stored matrices
constexpr int kThreads = 512;
constexpr int kPerSum = 8192;  // elements of a workgroup that sums squares

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

// The update from a gradient and the new momentum.
__device__ __forceinline__ float update_of(const Update &u, float g, float m) {
  return u.nesterov ? __builtin_fmaf(u.beta, m, g * u.grad_scale) : m;
}

// Workgroup (x, y): kPerSum elements of matrix y: the new momentum and the sum of the update's squares.
// In 64 bits, which hold the squares of every FP32 number.
template <bool kF32, bool kVector>
__global__ __launch_bounds__(256) void muon_momentum_kernel(const Update u, int64_t size, double *__restrict__ sums) {
  __shared__ double waves[4];
  double sum = 0.0;
  const int64_t base = blockIdx.y * size, end = base + size;
#pragma unroll
  for (int k = 0; k < kPerSum / 2048; ++k) {
    const int64_t at = base + static_cast<int64_t>(blockIdx.x) * kPerSum + k * 2048 + threadIdx.x * 8;
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
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    sums[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = (waves[0] + waves[1]) + (waves[2] + waves[3]);
}

// X in the workspace: hi + lo = kScale X, [mp][np], and hi transposed, [np][mp]; zeros in the padding.
struct Matrices {
  _Float16 *hi, *lo, *hit;
  int64_t mp, np;
};

__device__ __forceinline__ void split(float v, _Float16 &hi, _Float16 &lo) {
  hi = static_cast<_Float16>(v);
  lo = static_cast<_Float16>(v - static_cast<float>(hi));
}

// Workgroup (x, y, z): a tile of 64 x 64 of matrix z, [P][Q], rows 64 y.
template <bool kF32, bool kTall>
__global__ __launch_bounds__(256) void muon_start_kernel(const Update u, const double *__restrict__ sums, int count,
                                                         int64_t P, int64_t Q, const Matrices x) {
  __shared__ double waves[4];
  __shared__ float tile[64][65];
  double sum = 0.0;
  for (int i = threadIdx.x; i < count; i += 256) sum += sums[static_cast<int64_t>(blockIdx.z) * count + i];
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = (waves[0] + waves[1]) + (waves[2] + waves[3]);
  const double by = sum > 0.0 ? static_cast<double>(kScale) / sqrt(sum) : 0.0;

  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64, c0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int64_t base = blockIdx.z * P * Q;
  const int c = threadIdx.x & 63;
#pragma unroll 4
  for (int r = threadIdx.x >> 6; r < 64; r += 4) {
    float v = 0.0f;
    if (r0 + r < P && c0 + c < Q) {
      const int64_t at = base + (r0 + r) * Q + c0 + c;
      const float g = value_at<kF32>(u.grad, at);
      v = u.momentum != nullptr ? update_of(u, g, u.momentum[at]) : g;
      v = static_cast<float>(v * by);
    }
    tile[r][c] = v;
  }
  __syncthreads();
  // hi and lo by rows of X, then hi by its columns; 4 values per store
  const int64_t area = x.mp * x.np, at0 = blockIdx.z * area;
  const int64_t i0 = kTall ? c0 : r0, j0 = kTall ? r0 : c0;  // the tile's place in X
  const int q = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int r = threadIdx.x >> 4; r < 64; r += 16) {
    v4h hi, lo, hit;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      _Float16 h, l;
      split(kTall ? tile[q + k][r] : tile[r][q + k], h, l);
      hi[k] = h;
      lo[k] = l;
      hit[k] = static_cast<_Float16>(kTall ? tile[r][q + k] : tile[q + k][r]);
    }
    *reinterpret_cast<v4h *>(x.hi + at0 + (i0 + r) * x.np + j0 + q) = hi;
    *reinterpret_cast<v4h *>(x.lo + at0 + (i0 + r) * x.np + j0 + q) = lo;
    *reinterpret_cast<v4h *>(x.hit + at0 + (j0 + r) * x.mp + i0 + q) = hit;
  }
}

// ---------------------------------------------------------------------------------------
// Products.  A workgroup of 8 waves (4 x 2) makes a tile of kTile x kTile of P Q^T; each wave kTile / 4
// rows by kTile / 2 columns.  Stages of 64 K (128 bytes a row) of both operands go to LDS by
// buffer_load ... lds, double buffered: rows r and r + 8 of a group of 16 share a 256-byte line, the
// 16-byte chunks of a row are swapped by r mod 8, so that the 16 rows of a fragment read use all 64
// banks.  The operand with the output's columns is the instruction's first one: a lane then owns
// one output row and four consecutive columns.
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ int lds_pos(int row, int c) {
  const int r = row & 15;
  return (row >> 4) * 2048 + (r & 7) * 256 + (r >> 3) * 128 + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void *p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), static_cast<short>(0), static_cast<int>(bytes),
                                           0x00020000);
}

template <int kTile>
struct Tile {
  static constexpr int kM = kTile / 64, kN = kTile / 32;  // fragments of a wave
  v4f acc[kM][kN];
  int row, col;  // of the lane in the tile: + 16 i, + 16 j (then four columns)
};

// acc = rows [p, p + kTile) of P times rows [q, q + kTile) of Q; rows past the end count as zeros.  K % 128 == 0.
template <int kTile>
__device__ __forceinline__ void multiply(Tile<kTile> &t, const _Float16 *p, int64_t p_rows, const _Float16 *q,
                                         int64_t q_rows, int64_t K) {
  constexpr int kM = Tile<kTile>::kM, kN = Tile<kTile>::kN, kLoads = kTile / 64, kBytes = kTile * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t p0[kBytes], p1[kBytes], q0[kBytes], q1[kBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t ld = K * 2;
  const __amdgpu_buffer_rsrc_t rp = rsrc_of(p, (p_rows < kTile ? p_rows : kTile) * ld);
  const __amdgpu_buffer_rsrc_t rq = rsrc_of(q, (q_rows < kTile ? q_rows : kTile) * ld);
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int b = 8 * i + wave;  // 1 KB block: 4 lines of row group b / 2
    const int line = 4 * (b & 1) + (lane >> 4);
    off[i] = static_cast<uint32_t>(16 * (b >> 1) + line + 8 * ((lane >> 3) & 1)) * static_cast<uint32_t>(ld) +
             (((lane & 7) ^ line) << 4);
  }
  auto copy = [&](uint8_t *to_p, uint8_t *to_q, int64_t s) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (FP8Q_LDS void *)(to_p + (8 * i + wave) * 1024), 16,
                                               static_cast<int>(off[i]), static_cast<int>(s * 128), 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (FP8Q_LDS void *)(to_q + (8 * i + wave) * 1024), 16,
                                               static_cast<int>(off[i]), static_cast<int>(s * 128), 0, 0);
    }
  };
  const int r = lane & 15, kg = lane >> 4;
  const int at[2] = {lds_pos(r, kg), lds_pos(r, kg + 4)};
#pragma unroll
  for (int i = 0; i < kM; ++i)
#pragma unroll
    for (int j = 0; j < kN; ++j) t.acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto compute = [&](const uint8_t *from_p, const uint8_t *from_q) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v8h a[kM], b[kN];
#pragma unroll
      for (int i = 0; i < kM; ++i) a[i] = *reinterpret_cast<const v8h *>(from_p + (wm * kM + i) * 2048 + at[h]);
#pragma unroll
      for (int j = 0; j < kN; ++j) b[j] = *reinterpret_cast<const v8h *>(from_q + (wn * kN + j) * 2048 + at[h]);
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j) t.acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[j], a[i], t.acc[i][j], 0, 0, 0);
    }
  };
  // A wave waits for its own copies, then for the other waves: every copy of the stage has landed and
  // every wave has read the other buffer, which takes the next stage.
  auto meet = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  const int64_t stages = K / 64;  // even
  copy(p0, q0, 0);
  for (int64_t s = 0; s < stages; s += 2) {
    meet();
    copy(p1, q1, s + 1);
    compute(p0, q0);
    meet();
    if (s + 2 < stages) copy(p0, q0, s + 2);
    compute(p1, q1);
  }
  t.row = wm * (kTile / 4) + r;
  t.col = wn * (kTile / 2) + kg * 4;
}

// f(i, j) for every fragment of the lane: row t.row + 16 i, columns t.col + 16 j and the three after.
template <int kTile, class F>
__device__ __forceinline__ void each(const Tile<kTile> &t, F f) {
#pragma unroll
  for (int i = 0; i < Tile<kTile>::kM; ++i)
#pragma unroll
    for (int j = 0; j < Tile<kTile>::kN; ++j) f(t.row + 16 * i, t.col + 16 * j, t.acc[i][j]);
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

// kSquare false: A = X X^T and its diagonal; true: C = a I + b A + c A^2 from A and its diagonal.  Diagonals are
// unscaled and FP32, the matrices' own diagonals zero.
template <int kTile, bool kSquare>
__global__ __launch_bounds__(kThreads, kTile == 128 ? 4 : 2) void muon_symmetric_kernel(
    const _Float16 *__restrict__ from, int64_t K, int64_t mp, int G, const float *__restrict__ diagonal_in, Coefficients co,
    _Float16 *__restrict__ out, float *__restrict__ diagonal) {
  const int tiles = static_cast<int>((mp + kTile - 1) / kTile), per = tiles * (tiles + 1) / 2;
  const int64_t unit = unit_of(static_cast<int64_t>(per) * G);
  if (unit >= static_cast<int64_t>(per) * G) return;
  const int g = static_cast<int>(unit / per);
  int ti, tj;
  triangle(static_cast<int>(unit % per), ti, tj);
  const int64_t r0 = static_cast<int64_t>(ti) * kTile, c0 = static_cast<int64_t>(tj) * kTile;
  const _Float16 *x = from + g * mp * K;
  Tile<kTile> t;
  multiply<kTile>(t, x + r0 * K, mp - r0, x + c0 * K, mp - c0, K);
  _Float16 *const o = out + g * mp * mp;
  float *const d = diagonal + g * mp;
  const float *const d_in = kSquare ? diagonal_in + g * mp : nullptr;
  each<kTile>(t, [&](int row, int col, v4f v) {
    const int64_t i = r0 + row, j = c0 + col;
    if (i >= mp || j >= mp) return;
    v4h h;
    v4h a = {};
    v4f dj = {};
    float di = 0.0f;
    if (kSquare) {
      a = *reinterpret_cast<const v4h *>(x + i * mp + j);
      dj = *reinterpret_cast<const v4f *>(d_in + j);
      di = d_in[i];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float s = v[k] * (1.0f / kScale);
      if (i == j + k) {
        s *= 1.0f / kScale;
        d[i] = kSquare ? __builtin_fmaf(co.c, __builtin_fmaf(di, di, s), __builtin_fmaf(co.b, di, co.a)) : s;
        s = 0.0f;
      } else if (kSquare) {
        const float e = static_cast<float>(a[k]);
        s = __builtin_fmaf(co.c, __builtin_fmaf(di + dj[k], e, s), co.b * e);
      }
      h[k] = static_cast<_Float16>(s);
    }
    *reinterpret_cast<v4h *>(o + i * mp + j) = h;
    if (ti != tj) {
#pragma unroll
      for (int k = 0; k < 4; ++k) o[(j + k) * mp + i] = h[k];
    }
  });
}

struct Result {
  uint16_t *out;    // BF16 [G][P][Q], or null
  float *param;     // FP32 [G][P][Q]
  uint16_t *copy;   // BF16, the new param, or null
  const float *lr;  // device, or null
  float lr_host, decay, scale;
  int64_t P, Q;
};

// Tiles of C X.  Raster: 8 tiles of rows at a time, so that an XCD's run reads few panels.
__device__ __forceinline__ void raster(int u, int rows, int cols, int &i, int &j) {
  const int band = 8 * cols, first = u / band * 8;
  const int height = rows - first < 8 ? rows - first : 8;
  const int in = u % band;
  i = first + in % height;
  j = in / height;
}

// kLast false: X = C X in place and X^T into `hit`; true: the result, [P][Q].
template <int kTile, bool kLast, bool kTall>
__global__ __launch_bounds__(kThreads, kTile == 128 ? 4 : 2) void muon_apply_kernel(
    const _Float16 *__restrict__ c, const float *__restrict__ diagonal, const _Float16 *__restrict__ xt, const Matrices x,
    int G, const Result res) {
  const int64_t mp = x.mp, np = x.np;
  const int rows = static_cast<int>((mp + kTile - 1) / kTile), cols = static_cast<int>((np + kTile - 1) / kTile);
  const int64_t per = static_cast<int64_t>(rows) * cols, unit = unit_of(per * G);
  if (unit >= per * G) return;
  const int64_t g = unit / per;
  int ti, tj;
  raster(static_cast<int>(unit % per), rows, cols, ti, tj);
  const int64_t r0 = static_cast<int64_t>(ti) * kTile, c0 = static_cast<int64_t>(tj) * kTile;
  Tile<kTile> t;
  multiply<kTile>(t, c + g * mp * mp + r0 * mp, mp - r0, xt + g * mp * np + c0 * mp, np - c0, mp);
  _Float16 *const hi = x.hi + g * mp * np, *const lo = x.lo + g * mp * np, *const hit = x.hit + g * mp * np;
  const float *const d = diagonal + g * mp;
  const float lr = kLast && res.param != nullptr ? (res.lr != nullptr ? *res.lr : res.lr_host) : 0.0f;
  const float keep = 1.0f - lr * res.decay, step = lr * res.scale;
  const int64_t m = kTall ? res.Q : res.P, n = kTall ? res.P : res.Q;
  each<kTile>(t, [&](int row, int col, v4f v) {
    const int64_t i = r0 + row, j = c0 + col;
    if (i >= mp || j >= np) return;
    const v4h h0 = *reinterpret_cast<const v4h *>(hi + i * np + j), l0 = *reinterpret_cast<const v4h *>(lo + i * np + j);
    const float di = d[i];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = __builtin_fmaf(di, static_cast<float>(h0[k]) + static_cast<float>(l0[k]), v[k] * (1.0f / kScale));
    if constexpr (!kLast) {
      v4h h, l;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        _Float16 a, b;
        split(v[k], a, b);
        h[k] = a;
        l[k] = b;
        hit[(j + k) * mp + i] = a;
      }
      *reinterpret_cast<v4h *>(hi + i * np + j) = h;
      *reinterpret_cast<v4h *>(lo + i * np + j) = l;
    } else {
      if (i >= m) return;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (j + k >= n) break;
        const int64_t at = g * res.P * res.Q + (kTall ? (j + k) * res.Q + i : i * res.Q + j + k);
        const float o = v[k] * (1.0f / kScale);
        if (res.param == nullptr) {
          res.out[at] = static_cast<uint16_t>(pack2_bf16(o, 0.0f));
        } else {
          const float p = res.param[at] * keep - step * o;
          res.param[at] = p;
          if (res.copy != nullptr) res.copy[at] = static_cast<uint16_t>(pack2_bf16(p, 0.0f));
        }
      }
    }
  });
}

// The workspace: sums of squares, X (hi, lo), X^T twice, A, C and their diagonals.
struct Layout {
  int64_t G, P, Q, mp, np, count;  // count: workgroups that sum a matrix's squares
  int64_t sums, hi, lo, hit[2], a, c, da, dc, bytes;
  Layout(int64_t G, int64_t P, int64_t Q) : G(G), P(P), Q(Q) {
    mp = padded(P < Q ? P : Q);
    np = padded(P < Q ? Q : P);
    count = (P * Q + kPerSum - 1) / kPerSum;
    int64_t at = 0;
    auto take = [&](int64_t size) {
      const int64_t here = at;
      at += (size + 255) / 256 * 256;
      return here;
    };
    sums = take(8 * G * count);
    hi = take(2 * G * mp * np);
    lo = take(2 * G * mp * np);
    hit[0] = take(2 * G * mp * np);
    hit[1] = take(2 * G * mp * np);
    a = take(2 * G * mp * mp);
    c = take(2 * G * mp * mp);
    da = take(4 * G * mp);
    dc = take(4 * G * mp);
    bytes = at;
  }
};

// Tile size with the least time by rounds over the CUs.
template <class Units>
int tile_for(Units units, int64_t cus) {
  int best = 256;
  double least = 0;
  for (int tile : {256, 192, 128}) {
    const int64_t at_once = tile == 128 ? 2 * cus : cus;
    const double rounds = static_cast<double>((units(tile) + at_once - 1) / at_once) * (tile == 128 ? 2 : 1);
    const double time = rounds * tile * tile * (tile == 256 ? 1.0 : tile == 192 ? 1.1 : 1.4);
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
  else
    f(std::integral_constant<int, 128>{});
}

hipError_t run(const Layout &w, const Update &u, bool f32, const Coefficients &co, int64_t steps, const Result &res,
               void *workspace, hipStream_t stream) {
  uint8_t *const ws = static_cast<uint8_t *>(workspace);
  auto halves = [&](int64_t at) { return reinterpret_cast<_Float16 *>(ws + at); };
  auto floats = [&](int64_t at) { return reinterpret_cast<float *>(ws + at); };
  double *const sums = reinterpret_cast<double *>(ws + w.sums);
  const bool tall = w.P > w.Q, vector = w.P * w.Q % 8 == 0;
  const int64_t cus = device_cu_count();
  const int G = static_cast<int>(w.G);
  Matrices x = {halves(w.hi), halves(w.lo), halves(w.hit[0]), w.mp, w.np};

  {
    const dim3 grid(static_cast<uint32_t>(w.count), static_cast<uint32_t>(G)), block(256);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, u, w.P * w.Q, sums); };
    if (f32)
      vector ? go(muon_momentum_kernel<true, true>) : go(muon_momentum_kernel<true, false>);
    else
      vector ? go(muon_momentum_kernel<false, true>) : go(muon_momentum_kernel<false, false>);
    const dim3 tiles(static_cast<uint32_t>((tall ? w.mp : w.np) / 64), static_cast<uint32_t>((tall ? w.np : w.mp) / 64),
                     static_cast<uint32_t>(G));
    auto start = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, tiles, block, 0, stream, u, sums, static_cast<int>(w.count), w.P, w.Q, x);
    };
    if (f32)
      tall ? start(muon_start_kernel<true, true>) : start(muon_start_kernel<true, false>);
    else
      tall ? start(muon_start_kernel<false, true>) : start(muon_start_kernel<false, false>);
  }
  auto tiles = [](int64_t size, int tile) { return (size + tile - 1) / tile; };
  auto triangle_units = [&](int tile) { return w.G * tiles(w.mp, tile) * (tiles(w.mp, tile) + 1) / 2; };
  auto apply_units = [&](int tile) { return w.G * tiles(w.mp, tile) * tiles(w.np, tile); };
  const int sym = tile_for(triangle_units, cus), app = tile_for(apply_units, cus);
  auto grid_of = [](int64_t units) { return dim3(static_cast<uint32_t>((units + 7) / 8 * 8)); };
  for (int64_t s = 0; s < steps; ++s) {
    with_tile(sym, [&](auto tile) {
      constexpr int kT = decltype(tile)::value;
      hipLaunchKernelGGL((muon_symmetric_kernel<kT, false>), grid_of(triangle_units(kT)), dim3(kThreads), 0, stream, x.hi,
                         w.np, w.mp, G, nullptr, co, halves(w.a), floats(w.da));
      hipLaunchKernelGGL((muon_symmetric_kernel<kT, true>), grid_of(triangle_units(kT)), dim3(kThreads), 0, stream,
                         halves(w.a), w.mp, w.mp, G, floats(w.da), co, halves(w.c), floats(w.dc));
    });
    const _Float16 *const xt = halves(w.hit[s & 1]);
    x.hit = halves(w.hit[(s + 1) & 1]);
    with_tile(app, [&](auto tile) {
      constexpr int kT = decltype(tile)::value;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_of(apply_units(kT)), dim3(kThreads), 0, stream, halves(w.c), floats(w.dc), xt, x, G,
                           res);
      };
      if (s + 1 < steps)
        go(muon_apply_kernel<kT, false, false>);
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
  const int64_t rows = (w.mp + 127) / 128, cols = (w.np + 127) / 128;  // the smallest tiles
  return G <= 65535 && grid_fits(w.count, 256) && (P + 63) / 64 <= 65534 && grid_fits(w.np / 64, 256) &&
         rows * cols < (int64_t(1) << 30) / G && rows * rows < (int64_t(1) << 30) / G && grid_fits(G * rows * cols, kThreads) &&
         grid_fits(G * rows * rows, kThreads);
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
