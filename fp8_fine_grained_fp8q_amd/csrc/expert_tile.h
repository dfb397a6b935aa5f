// Tiles of 128 rows of expert-sorted rows, no tile across two experts: expert g's rows
// offsets[g] .. offsets[g+1]-1 (clamped to [0, M)) are cut into ceil(n_g / 128) tiles, and
// the experts' tiles follow each other.  Shared by the quantizers that write such tiles and
// the product that contracts over them.
//
// Each wave finds its expert from the offsets by itself, 64 experts per step, one per lane: no
// table in memory, no launch before the kernel.  An expert has fewer than 2^24 tiles, so 64 of
// them sum in 32 bits; the running total takes 64.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

// Inclusive prefix sum over the 64 lanes of a wave (all active): within rows of 16 lanes, then
// the rows' last lanes into the rows behind.
__device__ __forceinline__ int wave_prefix_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1, 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2, 3
  return v;
}

// The first row of expert g, clamped to [0, M], and its number of rows (none past the last expert).
__device__ __forceinline__ int expert_rows(const int32_t *__restrict__ offsets, int G, int64_t M, int g, int &count) {
  count = 0;
  if (g >= G) return 0;
  int64_t a = offsets[g], b = offsets[g + 1];
  a = a < 0 ? 0 : (a > M ? M : a);
  b = b < a ? a : (b > M ? M : b);
  count = static_cast<int>(b - a);
  return static_cast<int>(a);
}

// Tiles of n rows (n + 127 could pass 31 bits).
__device__ __forceinline__ int tiles_of(int n) { return n / 128 + (n % 128 != 0); }

// The first row and the number of rows (1 .. 128) of tile `tile`; false past the last tile.
// Every lane of the wave gets the same answer.
__device__ __forceinline__ bool expert_of_tile(const int32_t *__restrict__ offsets, int G, int64_t M, int64_t tile,
                                               int64_t &row, int &rows) {
  const int lane = threadIdx.x & 63;
  int64_t left = tile;  // tiles before it among the experts not yet passed
  for (int g0 = 0; g0 < G; g0 += 64) {
    int count;
    const int a = expert_rows(offsets, G, M, g0 + lane, count);
    const int tiles = tiles_of(count), incl = wave_prefix_sum(tiles);
    const uint64_t past = __ballot(incl > left);
    if (past != 0) {
      const int gl = __ffsll(static_cast<unsigned long long>(past)) - 1;
      const int skip = static_cast<int>(left) - __builtin_amdgcn_readlane(incl - tiles, gl);  // tiles of this expert
      row = static_cast<int64_t>(__builtin_amdgcn_readlane(a, gl)) + static_cast<int64_t>(skip) * 128;
      const int64_t rest = __builtin_amdgcn_readlane(count, gl) - static_cast<int64_t>(skip) * 128;
      rows = static_cast<int>(rest < 128 ? rest : 128);
      return true;
    }
    left -= __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// Expert g's first tile, its number of tiles and the rows of the last one (every lane the same
// answer).
__device__ __forceinline__ void tiles_of_expert(const int32_t *__restrict__ offsets, int G, int64_t M, int g,
                                                int64_t &first, int &tiles, int &rest) {
  const int lane = threadIdx.x & 63;
  first = 0;
  int own = 0;
  for (int g0 = 0; g0 <= g; g0 += 64) {  // g itself is counted with the last step, not before
    int count;
    expert_rows(offsets, G, M, g0 + lane, count);
    const int n = tiles_of(count), incl = wave_prefix_sum(g0 + lane < g ? n : 0);
    first += __builtin_amdgcn_readlane(incl, 63);
    if (g - g0 < 64) own = __builtin_amdgcn_readlane(count, g - g0);
  }
  tiles = tiles_of(own);
  rest = own - (tiles - 1) * 128;
}

}  // namespace fp8q
