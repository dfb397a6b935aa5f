// Weight gradients of MoE experts in E4M3, dW[g] = dY[g]^T X[g] for every local expert in one
// launch, for gfx950 (the pages' unified E4M3 format in the backward pass; see the dense
// weight-gradient product in gemm.hip).
//
//   C[g][p][q] = sum over expert g's token tiles b of
//                sa[b][p] * sb[b][q] * sum_{k in tile b} e4m3(aq[p][k]) * e4m3(bq[q][k])
//
// The contraction runs over the expert's tokens, in the tiles of 128 that
// quant_act_grouped_kernel writes (channel-major codes, one FP32 scale per tile and
// channel).  One v_mfma_f32_16x16x128_f8f6f4 covers one tile of a 16x16 block; it starts
// from zero and its result is scaled and added to an FP32 accumulator, acc = (P * sb) * sa +
// acc: two vector operations per element and token tile, as both scales vary inside a lane.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_tile.h"
#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
#define FP8Q_LDS __attribute__((address_space(3)))

// Buffer resource over `bytes` bytes at `p`; loads at or past the end return zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), static_cast<short>(0), static_cast<int>(bytes),
                                           0x00020000);
}

// LDS byte offset of the 16-byte chunk c (0..7) of operand row `row` in a stage.  A 16x16x128
// fragment is read as lane 16 kg + r taking chunks 2 kg and 2 kg + 1 of row r, so rows r and
// r + 8 of a group of 16 share a 256-byte line and the chunks of a row are XOR-swizzled by
// r mod 8: the 16 lanes of a read then touch every bank once.
__device__ __forceinline__ int chunk_pos(int row, int c) {
  const int r = row & 15;
  return (row >> 4) * 2048 + (r & 7) * 256 + (r >> 3) * 128 + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ v8i fragment(const FP8Q_LDS uint8_t *lds, int group, int lo, int hi) {
  const v4i a = *reinterpret_cast<const FP8Q_LDS v4i *>(lds + group * 2048 + lo);
  const v4i b = *reinterpret_cast<const FP8Q_LDS v4i *>(lds + group * 2048 + hi);
  return v8i{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// One workgroup of WM x WN waves computes a (16 FM WM) x (16 FN WN) tile of one expert's C,
// each wave 16 FM rows x 16 FN columns.  Stages of one token tile (operand codes and scales)
// are double buffered in LDS and filled by direct-to-LDS copies.
template <int WM, int WN, int FM, int FN>
struct Wgrad {
  static constexpr int kWaves = WM * WN;
  static constexpr int kTM = 16 * FM * WM, kTN = 16 * FN * WN;
  static constexpr int kA = kTM * 128, kB = kTN * 128;     // bytes of a stage's operands
  static constexpr int kScales = (kTM + kTN) * 4;          // and of its scales
  static constexpr int kStage = kA + kB + kScales;
  static constexpr int kCopiesA = kTM / 8 / kWaves, kCopiesB = kTN / 8 / kWaves;  // 1 KB copies per wave
  static constexpr int kScaleCopies = (kTM + kTN) / 64 / kWaves;
  static_assert(kTM % (8 * kWaves) == 0 && kTN % (8 * kWaves) == 0 && (kTM + kTN) % (64 * kWaves) == 0, "whole copies");
};

template <int WM, int WN, int FM, int FN>
__device__ __forceinline__ void wgrad_tile(const uint8_t *__restrict__ aq, const float *__restrict__ sa,
                                           const uint8_t *__restrict__ bq, const float *__restrict__ sb,
                                           const int32_t *__restrict__ offsets, int G, int64_t M, int64_t Mp, int P,
                                           int Q, void *__restrict__ c, int out_f32, FP8Q_LDS uint8_t *s0,
                                           FP8Q_LDS uint8_t *s1) {
  using W = Wgrad<WM, WN, FM, FN>;

  // Workgroups are dealt round-robin to the 8 XCDs; each XCD gets a contiguous run of tiles,
  // so that its L2 holds the panels that neighbouring tiles share.
  const int tp = (P + W::kTM - 1) / W::kTM, tq = (Q + W::kTN - 1) / W::kTN;
  const int total = gridDim.x, per = total / 8, rem = total % 8;
  const int xcd = blockIdx.x % 8, idx = blockIdx.x / 8;
  const int logical = xcd * per + (xcd < rem ? xcd : rem) + idx;
  const int g = logical / (tp * tq), in_g = logical - g * (tp * tq);
  const int64_t p0 = static_cast<int64_t>(in_g % tp) * W::kTM, q0 = static_cast<int64_t>(in_g / tp) * W::kTN;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, kg = lane >> 4;

  int64_t first64, tiles64;
  tiles_of_expert(offsets, G, M, g, first64, tiles64);
  // valid offsets never reach past the Mp / 128 tiles; others are kept inside the operands
  const int64_t end64 = first64 + tiles64 < Mp / 128 ? first64 + tiles64 : Mp / 128;
  const int tiles = __builtin_amdgcn_readfirstlane(static_cast<int>(end64 > first64 ? end64 - first64 : 0));
  const int first = __builtin_amdgcn_readfirstlane(static_cast<int>(tiles > 0 ? first64 : 0));

  const int rows_a = static_cast<int>(P - p0 < W::kTM ? P - p0 : W::kTM);
  const int rows_b = static_cast<int>(Q - q0 < W::kTN ? Q - q0 : W::kTN);
  const __amdgpu_buffer_rsrc_t ra = buffer_of(aq + p0 * Mp, rows_a * Mp);
  const __amdgpu_buffer_rsrc_t rb = buffer_of(bq + q0 * Mp, rows_b * Mp);

  // Copies: 1 KB block b of an operand holds 8 of a row group's 16 rows; lane l lands on line
  // 4 (b % 2) + l / 16, half (l / 8) % 2, slot l % 8 of group b / 2 (the inverse of chunk_pos).
  auto row_of = [&](int b, int &chunk) {
    const int line = 4 * (b & 1) + (lane >> 4);
    chunk = (lane & 7) ^ line;
    return 16 * (b >> 1) + line + 8 * ((lane >> 3) & 1);
  };
  int off_a[W::kCopiesA], off_b[W::kCopiesB];
#pragma unroll
  for (int i = 0; i < W::kCopiesA; ++i) {
    int chunk;
    const int row = row_of(i * W::kWaves + wave, chunk);
    off_a[i] = row * static_cast<int>(Mp) + chunk * 16;
  }
#pragma unroll
  for (int i = 0; i < W::kCopiesB; ++i) {
    int chunk;
    const int row = row_of(i * W::kWaves + wave, chunk);
    off_b[i] = row * static_cast<int>(Mp) + chunk * 16;
  }
  auto load = [&](int s, FP8Q_LDS uint8_t *st) {
    const int at = (first + s) * 128;
#pragma unroll
    for (int i = 0; i < W::kCopiesA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (FP8Q_LDS void *)(st + (i * W::kWaves + wave) * 1024), 16, off_a[i],
                                               at, 0, 0);
#pragma unroll
    for (int i = 0; i < W::kCopiesB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (FP8Q_LDS void *)(st + W::kA + (i * W::kWaves + wave) * 1024), 16,
                                               off_b[i], at, 0, 0);
    // scales: 64 of them per copy, first the tile's rows, then its columns; past the last row
    // or column nothing is read and zeros land
#pragma unroll
    for (int i = 0; i < W::kScaleCopies; ++i) {
      const int block = i * W::kWaves + wave;
      const bool is_a = block < W::kTM / 64;
      const int64_t tile = first + s;
      const int part = (is_a ? block : block - W::kTM / 64) * 64;
      const __amdgpu_buffer_rsrc_t r =
          buffer_of(is_a ? sa + tile * P + p0 : sb + tile * Q + q0, (is_a ? rows_a : rows_b) * 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (FP8Q_LDS void *)(st + W::kA + W::kB + block * 256), 4,
                                               (part + lane) * 4, 0, 0, 0);
    }
  };

  v4f acc[FM][FN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[f][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int lo = chunk_pos(l16, 2 * kg), hi = chunk_pos(l16, 2 * kg + 1);

  auto step = [&](const FP8Q_LDS uint8_t *cur, FP8Q_LDS uint8_t *next, int s) {
    // this wave's copies of stage s have landed; after the barrier every wave's have, and
    // every wave is done reading the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (s + 1 < tiles) load(s + 1, next);
    const FP8Q_LDS uint8_t *ca = cur, *cb = cur + W::kA, *cs = cur + W::kA + W::kB;
    v8i af[FM];
    float sr[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      af[f] = fragment(ca, wm * FM + f, lo, hi);
      sr[f] = *reinterpret_cast<const FP8Q_LDS float *>(cs + (wm * 16 * FM + f * 16 + l16) * 4);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const v8i bf = fragment(cb, wn * FN + j, lo, hi);
      const v4f sc =
          *reinterpret_cast<const FP8Q_LDS v4f *>(cs + (W::kTM + wn * 16 * FN + j * 16 + 4 * kg) * 4);
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
        const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf, af[f], zero, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][j][i] = __builtin_fmaf(part[i] * sc[i], sr[f], acc[f][j][i]);
      }
    }
  };

  if (tiles > 0) {
    load(0, s0);
    int s = 0;
    for (; s + 1 < tiles; s += 2) {
      step(s0, s1, s);
      step(s1, s0, s + 1);
    }
    if (s < tiles) step(s0, s1, s);
  }

  // Lane 16 kg + r owns row r and columns 4 kg .. 4 kg + 3 of each 16x16 block.
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    const int64_t p = p0 + wm * 16 * FM + f * 16 + l16;
    if (p >= P) continue;
    const int64_t base = (static_cast<int64_t>(g) * P + p) * Q;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int64_t q = q0 + wn * 16 * FN + j * 16 + 4 * kg;
      if (q >= Q) continue;
      const v4f v = acc[f][j];
      if (out_f32)
        *reinterpret_cast<v4f *>(static_cast<float *>(c) + base + q) = v;
      else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(c) + base + q) =
            make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
    }
  }
}

template <int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(64 * WM * WN, (WM * WN == 8 ? 1 : 2)) void wgrad_kernel(
    const uint8_t *__restrict__ aq, const float *__restrict__ sa, const uint8_t *__restrict__ bq,
    const float *__restrict__ sb, const int32_t *__restrict__ offsets, int G, int64_t M, int64_t Mp, int P, int Q,
    void *__restrict__ c, int out_f32) {
  __shared__ __attribute__((aligned(1024))) uint8_t stage0[Wgrad<WM, WN, FM, FN>::kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t stage1[Wgrad<WM, WN, FM, FN>::kStage];
  wgrad_tile<WM, WN, FM, FN>(aq, sa, bq, sb, offsets, G, M, Mp, P, Q, c, out_f32, (FP8Q_LDS uint8_t *)stage0,
                             (FP8Q_LDS uint8_t *)stage1);
}

namespace {

template <int WM, int WN, int FM, int FN>
hipError_t launch_tiles(const uint8_t *aq, const float *sa, const uint8_t *bq, const float *sb, const int32_t *offsets,
                        int64_t G, int64_t M, int64_t Mp, int64_t P, int64_t Q, void *c, bool out_f32,
                        hipStream_t stream) {
  using W = Wgrad<WM, WN, FM, FN>;
  const int64_t grid = G * ((P + W::kTM - 1) / W::kTM) * ((Q + W::kTN - 1) / W::kTN);
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((wgrad_kernel<WM, WN, FM, FN>), dim3(static_cast<uint32_t>(grid)), dim3(64 * WM * WN), 0, stream,
                     aq, sa, bq, sb, offsets, static_cast<int>(G), M, Mp, static_cast<int>(P), static_cast<int>(Q), c,
                     out_f32 ? 1 : 0);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_gemm_rowscaled(const uint8_t *aq, const float *sa, const uint8_t *bq, const float *sb,
                                         const int32_t *offsets, int64_t G, int64_t M, int64_t Mp, int64_t P,
                                         int64_t Q, void *c, bool out_f32, hipStream_t stream) {
  return launch_tiles<2, 2, 4, 4>(aq, sa, bq, sb, offsets, G, M, Mp, P, Q, c, out_f32, stream);
}

}  // namespace fp8q
