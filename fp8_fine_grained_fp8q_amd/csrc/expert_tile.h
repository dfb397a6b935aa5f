// Tiles of 128 rows of expert-sorted rows, no tile across two experts: expert g's rows
// offsets[g] .. offsets[g+1]-1 (clamped to [0, M)) are cut into ceil(n_g / 128) tiles, and
// the experts' tiles follow each other.  Shared by the quantizer that writes such tiles and
// the product that contracts over them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

// Inclusive prefix sum over the 64 lanes of a wave.
__device__ __forceinline__ int64_t wave_prefix_sum(int64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t u = __shfl_up(v, d);
    v += lane >= d ? u : 0;
  }
  return v;
}

// Clamped rows [a, b) of expert g, empty past the last expert.
__device__ __forceinline__ void expert_rows(const int32_t *__restrict__ offsets, int G, int64_t M, int g, int64_t &a,
                                            int64_t &b) {
  a = 0;
  b = 0;
  if (g >= G) return;
  a = offsets[g];
  b = offsets[g + 1];
  a = a < 0 ? 0 : (a > M ? M : a);
  b = b < a ? a : (b > M ? M : b);
}

// The first row and the number of rows (1 .. 128) of tile `tile`; false past the last tile.
// Every lane of the wave gets the same answer: 64 experts per step, one per lane.
__device__ __forceinline__ bool expert_of_tile(const int32_t *__restrict__ offsets, int G, int64_t M, int64_t tile,
                                               int64_t &row, int &rows) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int g0 = 0; g0 < G; g0 += 64) {
    int64_t a, b;
    expert_rows(offsets, G, M, g0 + lane, a, b);
    const int64_t tiles = (b - a + 127) / 128;
    const int64_t incl = before + wave_prefix_sum(tiles);
    const uint64_t past = __ballot(incl > tile);
    if (past != 0) {
      const int gl = __ffsll(static_cast<unsigned long long>(past)) - 1;
      const int64_t first = __shfl(incl - tiles, gl);
      const int64_t ga = __shfl(a, gl), gb = __shfl(b, gl);
      row = ga + (tile - first) * 128;
      rows = static_cast<int>(gb - row < 128 ? gb - row : 128);
      return true;
    }
    before = __shfl(incl, 63);
  }
  return false;
}

// Expert g's first tile, its number of tiles and the rows of the last one (every lane the same
// answer).
__device__ __forceinline__ void tiles_of_expert(const int32_t *__restrict__ offsets, int G, int64_t M, int g,
                                                int64_t &first, int64_t &tiles, int &rest) {
  const int lane = threadIdx.x & 63;
  int64_t sum = 0;
  for (int g0 = 0; g0 < g; g0 += 64) {
    int64_t a, b;
    expert_rows(offsets, g, M, g0 + lane, a, b);
    sum += (b - a + 127) / 128;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
  int64_t a, b;
  expert_rows(offsets, G, M, g, a, b);
  first = sum;
  tiles = (b - a + 127) / 128;
  rest = static_cast<int>(b - a - (tiles - 1) * 128);
}

}  // namespace fp8q
