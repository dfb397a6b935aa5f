// Weight gradients of MoE experts in E4M3, dW[g] = dY[g]^T X[g] for every local expert in one
// call, for gfx950 (the pages' unified E4M3 format in the backward pass; see the dense
// weight-gradient product in gemm.hip).
//
//   C[g][p][q] = sum over expert g's token tiles b of
//                sa[b][p] * sb[b][q] * sum_{k in tile b} e4m3(aq[p][k]) * e4m3(bq[q][k])
//
// The contraction runs over the expert's tokens, in the tiles of 128 that
// quant_act_grouped_kernel writes (one FP32 scale per tile and channel).  A tile's sum P starts
// from zero in the matrix core, which also forms the products of the scales, S = sa * sb, by an
// FP32 instruction of depth 1: each is one rounded product, and acc = P * S + acc is one vector
// operation per element and token tile, where both scales vary inside a lane and two were
// needed, (P * sa) * sb + acc (FP32 output 500 -> 488 us and 860 -> 838 us for the two sizes
// below).  S can pass FP32's range at either end where its term does not; waves watch the scales
// they meet and form such blocks again without it (ScaleRange, wide_products, wide_range_block; the
// watching costs 1 to 2 % of the cycles).
//
// BF16 output takes the FP8 matrix instructions.  Their sums of 64 products are off by 1.4e-5
// (2-norm, normal data, any of the shapes), far below BF16's rounding but above FP32's: FP32
// output widens the codes to BF16, exactly, and takes the BF16 instructions (8e-9), at half
// their rate.
//
// Two regimes, measured on one MI355X (product alone):
//  * few tokens per expert: the gradient's bytes.  32 experts of 4096 x 7168 over 8192 rows: FP32
//    850-870 us (4.4 TB/s of 3.76 GB), BF16 500-515 us.  Stores alone take 650 and 366 us, loads and
//    products alone about 700 and 450; the two overlap only in part.
//  * many: the matrix cores and the instructions around theirs.  4 experts of 7168 x 2048 over 16384
//    rows: BF16 245-250 us (1.9 PFLOP/s), FP32 435-450 us (1.1) by the wide kernel below; 289 and 483 us
//    by the small tiles.
//
// The kernel for few tokens: a workgroup of 8 waves computes 128 x 128 tiles of one expert, 32 x 64
// per wave in 32x32 blocks, two workgroups per CU, so that one's loads and stores run beside the
// other's products.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "expert_tile.h"
#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v32f __attribute__((ext_vector_type(32)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
#define FP8Q_LDS __attribute__((address_space(3)))

// Buffer resource over `bytes` bytes at `p`; loads at or past the end return zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), static_cast<short>(0), bytes, 0x00020000);
}

constexpr int kTile = 128;            // rows and columns of C per tile
constexpr int kWaves = 8;             // 4 x 2, 32 rows x 64 columns each
constexpr int kPanel = kTile * 128;   // bytes of one operand in a stage
constexpr int kScaleAt = 2 * kPanel;  // then 128 row scales and 128 column scales
constexpr int kStage = kScaleAt + 2 * kTile * 4;

// LDS byte offset of the 16-byte chunk c (0..7) of operand row `row` in a stage.  A fragment
// read takes one chunk of 32 rows per half wave; rows r and r + 8 of a group of 16 share a
// 256-byte line and the chunks of a row are XOR-swizzled by r mod 8, so that every 16 lanes
// of a read touch each bank once.
__device__ __forceinline__ int chunk_pos(int row, int c) {
  const int r = row & 15;
  return (row >> 4) * 2048 + (r & 7) * 256 + (r >> 3) * 128 + ((c ^ (r & 7)) << 4);
}

// Eight E4M3 codes as BF16 (exact).
__device__ __forceinline__ bf16x8 widen8(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ uint32_t lds_address(FP8Q_LDS uint8_t *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
}

__device__ __forceinline__ v8i join(const v4i &a, const v4i &b) {
  return v8i{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// LDS reads as single asm blocks that wait for themselves.  Written as C++ loads, the compiler
// has them wait for every direct-to-LDS copy that it cannot prove to be of other bytes, and
// with copies and stores of a varying number behind them that means vmcnt(0): each second
// stage then waited for the copies issued just before it and for the tile's stores (the copies
// that these reads do need are waited for at the stage's start).
template <int kAt>
__device__ __forceinline__ void read_chunks(v4i &a, v4i (&b)[2], uint32_t pa, uint32_t pb) {
  asm volatile(
      "ds_read_b128 %0, %3 offset:%5\n\tds_read_b128 %1, %4 offset:%6\n\tds_read_b128 %2, %4 offset:%7\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(a), "=&v"(b[0]), "=&v"(b[1])
      : "v"(pa), "v"(pb), "n"(kAt), "n"(kAt + kPanel), "n"(kAt + kPanel + 4096)
      : "memory");
}
template <int kAt>
__device__ __forceinline__ void read_chunks(v4i (&a)[2], v4i (&b)[2][2], uint32_t pa0, uint32_t pa1, uint32_t pb0,
                                            uint32_t pb1) {
  asm volatile(
      "ds_read_b128 %0, %6 offset:%10\n\tds_read_b128 %1, %7 offset:%10\n\t"
      "ds_read_b128 %2, %8 offset:%11\n\tds_read_b128 %3, %9 offset:%11\n\t"
      "ds_read_b128 %4, %8 offset:%12\n\tds_read_b128 %5, %9 offset:%12\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(a[0]), "=&v"(a[1]), "=&v"(b[0][0]), "=&v"(b[0][1]), "=&v"(b[1][0]), "=&v"(b[1][1])
      : "v"(pa0), "v"(pa1), "v"(pb0), "v"(pb1), "n"(kAt), "n"(kAt + kPanel), "n"(kAt + kPanel + 4096)
      : "memory");
}
// The scales of row l32 and of column 2 l32 + half of the wave.
template <int kAt>
__device__ __forceinline__ void read_scales(float &sr, float &sc, uint32_t pr, uint32_t pc) {
  asm volatile("ds_read_b32 %0, %2 offset:%4\n\tds_read_b32 %1, %3 offset:%5\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(sr), "=&v"(sc)
               : "v"(pr), "v"(pc), "n"(kAt), "n"(kAt + kTile * 4)
               : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Expert g's tiles of 128 tokens: the first one, their number and the tokens of the last one.  Valid
// offsets never reach past the last tile; others are kept inside the operands.
__device__ __forceinline__ void expert_tiles(const int32_t *offsets, int G, int64_t M, int64_t all_tiles, int g,
                                             int &first, int &tiles, int &rest) {
  int64_t first64;
  tiles_of_expert(offsets, G, M, g, first64, tiles, rest);
  const int64_t room = all_tiles - first64;
  tiles = room <= 0 ? 0 : (tiles < room ? tiles : static_cast<int>(room));
  first = tiles > 0 ? static_cast<int>(first64) : 0;
}

// The largest and smallest scales that a lane has met in a tile of C, as bits (which order like the values).
// If all are in [2^-63, 2^63] every product of two is a normal FP32 number.
struct ScaleRange {
  uint32_t top = 0u, low = ~0u;
  __device__ __forceinline__ void see(float a, float b) {
    top = max(top, max(__float_as_uint(a), __float_as_uint(b)));
    low = min(low, min(__float_as_uint(a), __float_as_uint(b)));
  }
  // of all lanes; also true for a scale of 0
  __device__ __forceinline__ bool wide() const {
    return __ballot(top > ((127u + 63u) << 23) || low < ((127u - 63u) << 23)) != 0;
  }
};

// Whether a product of one of kRows rows' scales and one of 64 columns' may not be a normal FP32 number, zeros
// aside: from the exponents of the largest and of the smallest of either, over all of an expert's tiles.
// For tiles with a scale of 0 or outside ScaleRange, of which it costs a tenth.
template <int kRows>
__device__ __forceinline__ bool wide_products(const float *sa, const float *sb, int64_t P, int64_t Q, int first, int tiles,
                                              int64_t row, int64_t col) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // keeps the addresses from being formed long before
  sa += static_cast<int64_t>(first) * P + row + (lane & (kRows - 1));
  sb += static_cast<int64_t>(first) * Q + col + lane;
  uint32_t tr = 0u, lr = ~0u, tc = 0u, lc = ~0u;  // the smallest ones less one: 0 wraps round past all others
#pragma unroll 4
  for (int t = 0; t < tiles; ++t, sa += P, sb += Q) {
    const uint32_t r = __float_as_uint(*sa), c = __float_as_uint(*sb);
    tr = max(tr, r);
    lr = min(lr, r - 1u);
    tc = max(tc, c);
    lc = min(lc, c - 1u);
  }
#pragma unroll 1
  for (int m = 32; m >= 1; m >>= 1) {
    tr = max(tr, static_cast<uint32_t>(__shfl_xor(static_cast<int>(tr), m)));
    lr = min(lr, static_cast<uint32_t>(__shfl_xor(static_cast<int>(lr), m)));
    tc = max(tc, static_cast<uint32_t>(__shfl_xor(static_cast<int>(tc), m)));
    lc = min(lc, static_cast<uint32_t>(__shfl_xor(static_cast<int>(lc), m)));
  }
  if (lr == ~0u || lc == ~0u) return false;  // all zeros
  // the largest is below 2^(e + 1), e the sum of two exponents, the smallest at least 2^e (subnormal: 2^-149)
  auto exponent = [](uint32_t bits) { return static_cast<int>(bits >> 23) - 127; };
  auto least = [&](uint32_t less_one) { return less_one < 0x7fffffu ? -149 : exponent(less_one + 1u); };
  return __builtin_amdgcn_readfirstlane(exponent(tr) + exponent(tc) > 125 || least(lr) + least(lc) < -126) != 0;
}

// Rows row .. row + 31 and columns col, col + 2 .. col + 62 of an expert's gradient, laid out as the wave's
// blocks, without the product of the scales: the smaller one multiplies a tile's sum, the larger
// one the result, so that nothing overflows that the term does not, and what underflows is below
// 2^-149 times the larger scale.  For scales that wide_products finds, which ordinary tensors do
// not have: straight from memory, two to nine times slower.
template <bool kOutF32>
__device__ __forceinline__ void wide_range_block(const uint8_t *aq, const float *sa, const uint8_t *bq, const float *sb,
                                                 int64_t P, int64_t Q, int first, int tiles, int64_t row, int64_t col,
                                                 v16f &acc) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // keeps the addresses from being formed long before
  const int l32 = lane & 31, half = lane >> 5;
  row += static_cast<int64_t>(first) * P;
  col += static_cast<int64_t>(first) * Q + 2 * l32;
  const uint8_t *a = aq + (row + l32) * 128 + 16 * half, *b = bq + col * 128 + 16 * half;
  sa += row + 4 * half;
  sb += col;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
#pragma unroll 1
  for (int t = 0; t < tiles; ++t, a += P * 128, b += Q * 128, sa += P, sb += Q) {
    v16f part = {};
    if constexpr (kOutF32) {
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        const v4i x = *reinterpret_cast<const v4i *>(a + 32 * m), y = *reinterpret_cast<const v4i *>(b + 32 * m);
#pragma unroll
        for (int r = 0; r < 4; r += 2)
          part = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8(x[r], x[r + 1]), widen8(y[r], y[r + 1]), part, 0, 0, 0);
      }
    } else {
#pragma unroll 1
      for (int m = 0; m < 4; m += 2) {
        const v4i *x = reinterpret_cast<const v4i *>(a + 32 * m), *y = reinterpret_cast<const v4i *>(b + 32 * m);
        part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(x[0], x[2]), join(y[0], y[2]), part, 0, 0, 0, 0, 0, 0);
      }
    }
    const float sc = *sb;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i % 4 == 0) __builtin_amdgcn_sched_barrier(0);  // few of the rows' scales at a time
      const float sr = sa[8 * (i >> 2) + (i & 3)];
      acc[i] = __builtin_fmaf(part[i] * fminf(sr, sc), fmaxf(sr, sc), acc[i]);
    }
  }
}

// The rows that are routed, offsets[G] of the M that there is room for.
__device__ __forceinline__ int routed_rows(const int32_t *offsets, int G, int64_t M) {
  const int n = offsets[G];
  return n < 0 ? 0 : (n > M ? static_cast<int>(M) : n);
}

// The tile row p and the run of tile columns r of expert g that unit `unit` computes, of tp
// rows and `runs` runs; false for units past an expert's last run.  Workgroups are dealt
// round-robin to the 8 XCDs, and a grid of several units per workgroup is a multiple of 8.  Each XCD gets a contiguous eighth of every expert's runs, four rows
// of tiles at a time, column by column: neighbouring workgroups share operands in their L2 and
// write neighbouring parts of the same rows, and experts of different sizes load all XCDs alike
// (whole experts per XCD: 8 uneven experts of 7168 x 2048 over 16384 rows FP32 548 us instead of 496,
// BF16 294 instead of 277).
__device__ __forceinline__ bool place(uint32_t unit, int tp, int runs, int &g, int &p, int &r) {
  const int per = (tp * runs + 7) / 8;
  const int xcd = static_cast<int>(unit % 8), idx = static_cast<int>(unit / 8);
  g = idx / per;
  const int in_g = xcd * per + idx % per;
  if (in_g >= tp * runs) return false;
  const int span = 4 * runs, first = in_g / span * 4, high = tp - first < 4 ? tp - first : 4, in_s = in_g % span;
  p = first + in_s % high;
  r = in_s / high;
  return true;
}

// C tiles (p0, q) for the run of 128-column tiles q0 .. q0 + 128 (count - 1) of expert g.
template <bool kOutF32>
__device__ __forceinline__ void wgrad_run(const uint8_t *__restrict__ aq, const float *__restrict__ sa,
                                          const uint8_t *__restrict__ bq, const float *__restrict__ sb,
                                          const int32_t *__restrict__ offsets, int G, int64_t M, int64_t all_tiles,
                                          int64_t P, int64_t Q, int g, int64_t p0, int64_t q0, int count,
                                          void *__restrict__ c, FP8Q_LDS uint8_t *st) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, half = lane >> 5;

  int first, tiles, rest;
  expert_tiles(offsets, G, M, all_tiles, g, first, tiles, rest);
  const int last = (rest + 31) / 32;

  // Copies: an operand's 16 KB stage is contiguous in memory.  1 KB block b = 8 i + wave of it
  // in LDS holds 8 of a row group's 16 rows; lane l lands on line 4 (b % 2) + l / 16, half (l / 8)
  // % 2, slot l % 8 of group b / 2 (the inverse of chunk_pos), on row 64 i + at.  For the
  // columns' operand, row 64 w + 32 n + l in LDS is column 64 w + 2 l + n: a lane's elements of a
  // wave's two column blocks are then neighbours in memory.
  const int line = 4 * (wave & 1) + (lane >> 4);
  const int at = 16 * (wave >> 1) + line + 8 * ((lane >> 3) & 1), chunk = ((lane & 7) ^ line) * 16;
  const int off_a = at * 128 + chunk, off_b = (at & 31) * 256 + (at >> 5) * 128 + chunk;
  auto load = [&](int j, int s, FP8Q_LDS uint8_t *st) {
    const int64_t at_a = static_cast<int64_t>(first + s) * P + p0;
    const int64_t at_b = static_cast<int64_t>(first + s) * Q + q0 + j * kTile;
    const __amdgpu_buffer_rsrc_t ra = buffer_of(aq + at_a * 128, kPanel), rb = buffer_of(bq + at_b * 128, kPanel);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      FP8Q_LDS uint8_t *to = st + (kWaves * i + wave) * 1024;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (FP8Q_LDS void *)to, 16, off_a, i * 8192, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (FP8Q_LDS void *)(to + kPanel), 16, off_b, i * 8192, 0, 0);
    }
    // waves 0 and 1 copy 64 of the rows' scales each, waves 2 and 3 of the columns'
    if (wave >= 4) return;
    const __amdgpu_buffer_rsrc_t rs = buffer_of((wave < 2 ? sa + at_a : sb + at_b) + (wave & 1) * 64, 256);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (FP8Q_LDS void *)(st + kScaleAt + wave * 256), 4, lane * 4, 0, 0, 0);
  };

  // Element i of block n is row 8 (i / 4) + 4 half + i % 4, column 2 l32 + n of the wave.
  v16f acc[2];
  ScaleRange range;
  auto clear = [&]() {
    range = ScaleRange();
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][i] = 0.0f;
  };
  // Each store writes two whole rows of 64 columns: full 128-byte lines, which the streaming
  // stores need (with half lines the FP32 gradient of 32 experts x 4096 x 7168 took 1.3 ms, with
  // whole ones and ordinary stores 1.4 ms).
  constexpr int kSize = kOutF32 ? 4 : 2, kStream = 2;  // bytes of an element; the streaming-store flag
  const int64_t c0 = (static_cast<int64_t>(g) * P + p0 + wm * 32) * Q + q0 + wn * 64;
  const int ld = static_cast<int>(Q) * kSize, off_c = 4 * half * ld + 2 * l32 * kSize;
  auto store = [&](int j) {
    const __amdgpu_buffer_rsrc_t rc = buffer_of(static_cast<uint8_t *>(c) + (c0 + j * kTile) * kSize, 32 * ld);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = (8 * (i >> 2) + (i & 3)) * ld;
      if (kOutF32)
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(acc[0][i]), __float_as_uint(acc[1][i])}, rc, off_c,
                                              row, kStream);
      else
        __builtin_amdgcn_raw_buffer_store_b32(pack2_bf16(acc[0][i], acc[1][i]), rc, off_c, row, kStream);
    }
  };
  clear();
  if (tiles == 0) {
    for (int j = 0; j < count; ++j) store(j);
    return;
  }

  // LDS addresses, in the first stage, of the lane's rows' chunk 2 m + half: chunks 2 m and 2 m + 1
  // hold the tokens 32 m .. 32 m + 31.
  uint32_t at_a[4], at_b[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint32_t pos = lds_address(st) + chunk_pos(l32, 2 * m + half);
    at_a[m] = pos + wm * 4096;
    at_b[m] = pos + wn * 8192;
  }
  const uint32_t at_sr = lds_address(st) + kScaleAt + (wm * 32 + l32) * 4;
  const uint32_t at_sc = lds_address(st) + kScaleAt + (wn * 64 + 2 * l32 + half) * 4;
  // Waits for the LDS reads and then for the other waves.  Not __syncthreads(), whose fence would
  // wait for the copies and stores in flight.
  auto meet = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stages run through the run's tiles without a break.  A wave's copies and stores complete in
  // the order of their issue, so a copy behind a tile's stores would wait for those to drain:
  // at the end of a tile the copies of the next two stages are issued first, and a stage's start
  // waits for no more than the operations behind its own copies allow (at least kCopies, five in
  // waves 0-3, and kStores).
  constexpr int kStores = 16, kCopies = 4;
  int j = 0, s = 0;          // the stage being multiplied
  bool ahead = false;        // the next stage's copies are issued already
  int stores = 0;            // 2: a tile ended a stage ago; 1: two stages ago
  uint32_t redo = 0;         // the run's tiles (at most 4) with scales outside the range, or of 0
  auto stage = [&](auto parity) {
    constexpr int kCur = decltype(parity)::value * kStage;  // the stage's place in LDS
    FP8Q_LDS uint8_t *cur = st + kCur, *next = st + (kStage - kCur);
    if (stores == 2 && ahead)
      wait_loads<kStores + kCopies>();
    else if (stores != 0)
      wait_loads<kStores>();
    else
      wait_loads<0>();
    meet();  // every wave's copies have landed, and every wave has read the other buffer
    const bool ends = s + 1 == tiles;
    int jn = j, sn = s;
    auto advance = [&]() {
      const bool wrap = sn + 1 == tiles;
      jn += wrap ? 1 : 0;
      sn = wrap ? 0 : sn + 1;
      return jn < count;
    };
    const bool more = advance();
    const int j1 = jn, s1 = sn;
    if (more && !ahead) load(jn, sn, next);
    stores = stores == 2 && ahead ? 1 : 0;
    ahead = false;
    const int used = ends ? last : 4;  // the 32-token parts of the tile that hold tokens
    v16f part[2] = {};
    if constexpr (kOutF32) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m > 0 && m >= used) break;
        v4i a, b[2];
        read_chunks<kCur>(a, b, at_a[m], at_b[m]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const bf16x8 wa = widen8(a[2 * r], a[2 * r + 1]);
#pragma unroll
          for (int n = 0; n < 2; ++n)
            part[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wa, widen8(b[n][2 * r], b[n][2 * r + 1]), part[n], 0, 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h > 0 && used <= 2) break;
        v4i a[2], b[2][2];
        read_chunks<kCur>(a, b, at_a[2 * h], at_a[2 * h + 1], at_b[2 * h], at_b[2 * h + 1]);
#pragma unroll
        for (int n = 0; n < 2; ++n)
          part[n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(a[0], a[1]), join(b[n][0], b[n][1]), part[n], 0,
                                                                    0, 0, 0, 0, 0);
      }
    }
    float sr, sc;
    read_scales<kCur>(sr, sc, at_sr, at_sc);
    const v32f scale = __builtin_amdgcn_mfma_f32_32x32x1f32(sr, sc, v32f{}, 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    range.see(sr, sc);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][i] = __builtin_fmaf(part[n][i], scale[16 * n + i], acc[n][i]);
    if (ends) {
      if (more) {
        meet();  // every wave has read this stage too: its buffer takes the stage after the next
        if (advance()) {
          load(jn, sn, cur);
          ahead = true;
        }
      }
      redo |= range.wide() ? 1u << j : 0u;
      store(j);
      clear();
      stores = 2;
    }
    j = j1;
    s = s1;
    return more;
  };
  load(0, 0, st);
  while (stage(std::integral_constant<int, 0>{}) && stage(std::integral_constant<int, 1>{})) {
  }
  if (redo == 0) return;
  wait_loads<0>();  // the tiles' first stores
  for (j = 0; j < count; ++j) {
    const int64_t row = p0 + wm * 32, col = q0 + j * kTile + wn * 64;
    if ((redo >> j & 1u) == 0 || !wide_products<32>(sa, sb, P, Q, first, tiles, row, col)) continue;
#pragma unroll
    for (int n = 0; n < 2; ++n)
      wide_range_block<kOutF32>(aq, sa, bq, sb, P, Q, first, tiles, row, col + n, acc[n]);
    store(j);
  }
}

// Leaves if the routed rows make `deepest` token tiles of an expert or more on average (0: never).
template <bool kOutF32>
__global__ __launch_bounds__(64 * kWaves, 4) void wgrad_kernel(
    const uint8_t *__restrict__ aq, const float *__restrict__ sa, const uint8_t *__restrict__ bq,
    const float *__restrict__ sb, const int32_t *__restrict__ offsets, int G, int64_t M, int64_t all_tiles, int P,
    int Q, int run, int deepest, void *__restrict__ c) {
  __shared__ __attribute__((aligned(1024))) uint8_t stages[2 * kStage];
  if (deepest > 0 && routed_rows(offsets, G, M) >= deepest * (int64_t(kTile) * G)) return;
  const int tp = P / kTile, tq = Q / kTile;
  int g, p, r;
  if (!place(blockIdx.x, tp, (tq + run - 1) / run, g, p, r)) return;
  const int q = r * run;
  wgrad_run<kOutF32>(aq, sa, bq, sb, offsets, G, M, all_tiles, P, Q, g, static_cast<int64_t>(p) * kTile,
                     static_cast<int64_t>(q) * kTile, tq - q < run ? tq - q : run, c, (FP8Q_LDS uint8_t *)stages);
}

// ---------------------------------------------------------------------------------------
// The kernel for many tokens: tiles of 256 x 128, 64 x 64 per wave (4 x 2 waves), one workgroup per
// CU.  The two waves of a SIMD (w and w + 4) take turns: one multiplies a token tile from registers
// while the other scales and adds its last one and reads the next from LDS.  Against the 128 x 128
// tiles a quarter less is copied, and a third less read from LDS and widened per product.
//
// 4 experts of 7168 x 2048 over 16384 rows: BF16 289 -> 242 us, FP32 483 -> 432 us.  BF16 takes 456
// to 467 thousand cycles.  The matrix cores work in 62 to 64 % of them; the vector instructions, 79 per wave and token
// tile and 64 of them the promotion, issue once per 8 cycles beside FP8 products and fill up to 80 %;
// a tile's start and end are 4 us of 36.  On codes of zeros it takes 196 us: the clock is higher then.  FP32 is bound by the issue
// of the widening: 315 us without the products, 307 without the widening.  Three things it needed: no
// branch and no address arithmetic between the barriers (BF16 310 us with them), the copies behind the
// matrix instructions and not behind the reads, and no instruction that waits for a matrix result
// right before another matrix instruction (265 -> 250 us).
// ---------------------------------------------------------------------------------------
constexpr int kWideRows = 256;
constexpr int kWideScaleAt = kWideRows * 128 + kPanel;  // then the rows' scales and the columns'
constexpr int kWideStage = kWideScaleAt + 8 * 256;  // waves 6 and 7 copy what 4 and 5 copy, behind it
constexpr int kRing = 3;  // stages in LDS: one read, two in flight

// A wave's operands of a stage and the scales of its row `lane` and of columns 2 l32, 2 l32 + 1.
// a[f][m], b[n][m]: chunk 2 m + half of row 32 f + l32 and column block n.
__device__ __forceinline__ void read_stage(v4i (&a)[2][4], v4i (&b)[2][4], float &sr, f32x2 &sc, const uint32_t (&pa)[4],
                                           const uint32_t (&pb)[4], uint32_t pr, uint32_t pc) {
  asm volatile(
      "ds_read_b32 %16, %26\n\tds_read_b64 %17, %27\n\t"
      "ds_read_b128 %0, %18\n\tds_read_b128 %8, %22\n\tds_read_b128 %1, %19\n\tds_read_b128 %9, %23\n\t"
      "ds_read_b128 %4, %18 offset:4096\n\tds_read_b128 %5, %19 offset:4096\n\t"
      "ds_read_b128 %2, %20\n\tds_read_b128 %10, %24\n\tds_read_b128 %3, %21\n\tds_read_b128 %11, %25\n\t"
      "ds_read_b128 %6, %20 offset:4096\n\tds_read_b128 %7, %21 offset:4096\n\t"
      "ds_read_b128 %12, %22 offset:4096\n\tds_read_b128 %13, %23 offset:4096\n\t"
      "ds_read_b128 %14, %24 offset:4096\n\tds_read_b128 %15, %25 offset:4096\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[0][2]), "=&v"(a[0][3]), "=&v"(a[1][0]), "=&v"(a[1][1]),
        "=&v"(a[1][2]), "=&v"(a[1][3]), "=&v"(b[0][0]), "=&v"(b[0][1]), "=&v"(b[0][2]), "=&v"(b[0][3]),
        "=&v"(b[1][0]), "=&v"(b[1][1]), "=&v"(b[1][2]), "=&v"(b[1][3]), "=&v"(sr), "=&v"(sc)
      : "v"(pa[0]), "v"(pa[1]), "v"(pa[2]), "v"(pa[3]), "v"(pb[0]), "v"(pb[1]), "v"(pb[2]), "v"(pb[3]), "v"(pr), "v"(pc)
      : "memory");
}

template <bool kOutF32>
__device__ __forceinline__ void wgrad_wide_run(const uint8_t *__restrict__ aq, const float *__restrict__ sa,
                                               const uint8_t *__restrict__ bq, const float *__restrict__ sb,
                                               const int32_t *__restrict__ offsets, int G, int64_t M, int64_t all_tiles,
                                               int64_t P, int64_t Q, int g, int64_t p0, int64_t q0,
                                               void *__restrict__ c, FP8Q_LDS uint8_t *st) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, half = lane >> 5;
  const bool lead = wave < 4;

  int first, tiles, rest;
  expert_tiles(offsets, G, M, all_tiles, g, first, tiles, rest);

  // Copies, as in wgrad_run: wave w moves 1 KB block 8 i + w of either operand.  parts: 64-row parts of
  // the tile that C has; the last tile of a P of 128 modulo 256 copies its rows twice and stores
  // them once.
  const int line = 4 * (wave & 1) + (lane >> 4);
  const int at = 16 * (wave >> 1) + line + 8 * ((lane >> 3) & 1), chunk = ((lane & 7) ^ line) * 16;
  const int off_a = at * 128 + chunk, off_b = (at & 31) * 256 + (at >> 5) * 128 + chunk;
  const int parts = P - p0 < kWideRows ? 2 : 4;
  const uint8_t *from_a = aq + (static_cast<int64_t>(first) * P + p0) * 128;
  const uint8_t *from_b = bq + (static_cast<int64_t>(first) * Q + q0) * 128;
  const float *from_s = wave < 4 ? sa + static_cast<int64_t>(first) * P + p0 + (wave & (parts - 1)) * 64
                                 : sb + static_cast<int64_t>(first) * Q + q0 + (wave & 1) * 64;
  const int64_t step_a = P * 128, step_b = Q * 128, step_s = wave < 4 ? P : Q;
  int copied = 0;                           // stages
  FP8Q_LDS uint8_t *to = st + wave * 1024;  // where the next one goes
  // Copy i of 7 of the next stage.  Past the last stage the copies go through empty resources (zeros,
  // no traffic), so that every wave always has the same number in flight.
  auto copy = [&](int i) {
    const bool some = copied < tiles;
    if (i < 4)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(from_a, some ? parts * 8192 : 0), (FP8Q_LDS void *)(to + i * 8192),
                                               16, off_a, (i & (parts - 1)) * 8192, 0, 0);
    else if (i < 6)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(from_b, some ? kPanel : 0), (FP8Q_LDS void *)(to + i * 8192), 16,
                                               off_b, (i - 4) * 8192, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(from_s, some ? 256 : 0),
                                               (FP8Q_LDS void *)(to + kWideScaleAt - wave * 768), 4, lane * 4, 0, 0, 0);
  };
  auto turn = [&]() {
    ++copied;
    from_a += step_a;
    from_b += step_b;
    from_s += step_s;
    to = to == st + wave * 1024 + (kRing - 1) * kWideStage ? st + wave * 1024 : to + kWideStage;
  };
  auto copy_stage = [&]() {
#pragma unroll
    for (int i = 0; i < 7; ++i) copy(i);
  };

  // Element i of block (f, n) is row 32 f + 8 (i / 4) + 4 half + i % 4, column 2 l32 + n of the wave.
  v16f acc[2][2], part[2][2];
  auto clear = [&](v16f (&x)[2][2]) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[f][n][i] = 0.0f;
  };
  const bool mine = wm < parts;  // this wave's rows are in C
  const int64_t c0 = (static_cast<int64_t>(g) * P + p0 + wm * 64) * Q + q0 + wn * 64;
  constexpr int kSize = kOutF32 ? 4 : 2, kStream = 2;  // bytes of an element; the streaming-store flag
  const int ld = static_cast<int>(Q) * kSize, off_c = 4 * half * ld + 2 * l32 * kSize;
  auto store = [&]() {
    if (!mine) return;
    const __amdgpu_buffer_rsrc_t rc = buffer_of(static_cast<uint8_t *>(c) + c0 * kSize, 64 * ld);
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = (32 * f + 8 * (i >> 2) + (i & 3)) * ld;
        if (kOutF32)
          __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(acc[f][0][i]), __float_as_uint(acc[f][1][i])}, rc,
                                                off_c, row, kStream);
        else
          __builtin_amdgcn_raw_buffer_store_b32(pack2_bf16(acc[f][0][i], acc[f][1][i]), rc, off_c, row, kStream);
      }
  };
  clear(acc);
  clear(part);
  if (tiles == 0) {
    store();
    return;
  }

  // LDS address, in the first stage, of the lane's row's chunk `half`; chunk 2 m + half is at ^ 32 m.
  const uint32_t at_0 = lds_address(st) + chunk_pos(l32, half);
  uint32_t at_sr = lds_address(st) + kWideScaleAt + (wm * 64 + lane) * 4;
  uint32_t at_sc = lds_address(st) + kWideScaleAt + (kWideRows + wn * 64 + 2 * l32) * 4;
  auto barrier = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // Phases end at a barrier.  The lead waves 0-3 run one ahead: in phase 2 t they read stage t, in phase
  // 2 t + 1 they multiply it, while the others read it.  Stage t is last read in phase 2 t + 1 and its
  // place free from phase 2 t + 2 on, where the others multiply it and copy stage t + 3; the lead
  // waves, which multiply it in phase 2 t + 1, copy stage t + 2 there.  A wave waits at the end of its
  // products for all but the copies that it just issued: the lead waves' of stage t + 1 have then
  // landed at the end of phase 2 t + 1, the others' of stage t + 2 at the end of phase 2 t + 2, both before
  // those stages are first read (phases 2 t + 2 and 2 t + 4).
  copy_stage();
  turn();
  copy_stage();
  if (lead) {
    wait_loads<7>();
    barrier();
  } else {
    turn();
    copy_stage();
    wait_loads<14>();
    barrier();
    wait_loads<7>();
    barrier();
  }
  // Column block n's sums, part[.][n], are scaled and added in the next reading phase, with BF16 output
  // block 0's beside block 1's products.
  ScaleRange range;
  int cur = 0;           // the stage's place in LDS
  v32f scale[2] = {};    // of column block n; BF16 output keeps one at a time, in scale[1]
  auto add = [&](int n, const v32f &by, int from, int to) {
#pragma unroll
    for (int i = from; i < to; ++i)
      acc[i / 16][n][i % 16] = __builtin_fmaf(part[i / 16][n][i % 16], by[i], acc[i / 16][n][i % 16]);
  };
  auto scales = [&](float sr, float sc) { return __builtin_amdgcn_mfma_f32_32x32x1f32(sr, sc, v32f{}, 0, 0, 0); };
  // The order of a phase as written: the value is taken as changed here.
  auto pin = []() { __builtin_amdgcn_sched_barrier(0); };
  auto pinned = [](auto &x) {
    asm volatile("" : "+v"(x));
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int t = 0; t < tiles; ++t) {
    turn();
    if (kOutF32) add(0, scale[0], 0, 32);
    add(1, scale[1], 0, 32);
    asm volatile("" : "+v"(acc[0][0]), "+v"(acc[1][0]), "+v"(acc[0][1]), "+v"(acc[1][1]));
    v4i a[2][4], b[2][4];
    float sr;
    f32x2 sc;
    const uint32_t a0 = at_0 + (cur + wm * 8192), b0 = at_0 + (cur + kWideRows * 128 + wn * 8192);
    const uint32_t pa[4] = {a0, a0 ^ 32, a0 ^ 64, a0 ^ 96}, pb[4] = {b0, b0 ^ 32, b0 ^ 64, b0 ^ 96};
    read_stage(a, b, sr, sc, pa, pb, at_sr + cur, at_sc + cur);
    cur = cur == (kRing - 1) * kWideStage ? 0 : cur + kWideStage;
    const v16f zero = {};
    if constexpr (kOutF32) {
      // Steps of 16 tokens: four products each, and behind every one the widening of a quarter of
      // the next step's operands.
      bf16x8 wide[2][4];  // of two steps: row blocks 0 and 1, column blocks 0 and 1
      auto widen = [&](int step, int k) {
        const v4i &x = k < 2 ? a[k][step >> 1] : b[k - 2][step >> 1];
        const int r = 2 * (step & 1);
        wide[step & 1][k] = widen8(x[r], x[r + 1]);
      };
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        widen(0, k);
        pinned(wide[0][k]);
      }
      barrier();
#pragma unroll
      for (int step = 0; step < 8; ++step)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int f = k >> 1, n = k & 1;
          part[f][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wide[step & 1][f], wide[step & 1][2 + n],
                                                               step == 0 ? zero : part[f][n], 0, 0, 0);
          pinned(part[f][n]);
          if (step < 7) {
            widen(step + 1, k);
            pinned(wide[(step + 1) & 1][k]);
            if (k == 0) copy(step);
            if (step == 0 && k == 1) range.see(sr, half ? sc.y : sc.x);
            pin();
          }
        }
      scale[0] = scales(sr, sc.x);
      pinned(scale[0]);
      scale[1] = scales(sr, sc.y);
      pinned(scale[1]);
    } else {
      barrier();
      auto multiply = [&](int n, int f, int h, const v16f &sum) {
        part[f][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(a[f][2 * h], a[f][2 * h + 1]),
                                                                     join(b[n][2 * h], b[n][2 * h + 1]), sum, 0, 0, 0, 0,
                                                                     0, 0);
        pinned(part[f][n]);
      };
      multiply(0, 0, 0, zero);
      copy(0);
      copy(1);
      pin();
      multiply(0, 0, 1, part[0][0]);
      copy(2);
      copy(3);
      pin();
      multiply(0, 1, 0, zero);
      copy(4);
      copy(5);
      pin();
      multiply(0, 1, 1, part[1][0]);
      scale[1] = scales(sr, sc.x);
      pinned(scale[1]);
      multiply(1, 0, 0, zero);
      copy(6);
      pin();
      multiply(1, 0, 1, part[0][1]);
      add(0, scale[1], 0, 8);
      pin();
      multiply(1, 1, 0, zero);
      add(0, scale[1], 8, 20);
      pin();
      multiply(1, 1, 1, part[1][1]);
      range.see(sr, half ? sc.y : sc.x);
      add(0, scale[1], 20, 32);
      pin();
      scale[1] = scales(sr, sc.y);
      pinned(scale[1]);
    }
    wait_loads<7>();
    barrier();
  }
  if (lead) barrier();
  wait_loads<0>();
  if (kOutF32) add(0, scale[0], 0, 32);
  add(1, scale[1], 0, 32);
  const int64_t row = p0 + wm * 64, col = q0 + wn * 64;
  if (mine && range.wide() && wide_products<64>(sa, sb, P, Q, first, tiles, row, col)) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      wide_range_block<kOutF32>(aq, sa, bq, sb, P, Q, first, tiles, row + 32 * (k >> 1), col + (k & 1), acc[k >> 1][k & 1]);
  }
  store();
}

// Leaves if the routed rows make fewer than `deepest` token tiles of an expert on average.  A workgroup
// takes every gridDim.x-th tile, so that few of them have to leave.
template <bool kOutF32>
__global__ __launch_bounds__(64 * kWaves, 2) void wgrad_wide_kernel(
    const uint8_t *__restrict__ aq, const float *__restrict__ sa, const uint8_t *__restrict__ bq,
    const float *__restrict__ sb, const int32_t *__restrict__ offsets, int G, int64_t M, int64_t all_tiles, int P,
    int Q, int deepest, void *__restrict__ c) {
  __shared__ __attribute__((aligned(1024))) uint8_t stages[kRing * kWideStage];
  if (routed_rows(offsets, G, M) < deepest * (int64_t(kTile) * G)) return;
  const int tp = (P + kWideRows - 1) / kWideRows, tq = Q / kTile, units = 8 * G * ((tp * tq + 7) / 8);
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    int g, p, q;
    if (!place(u, tp, tq, g, p, q)) continue;
    // its last barrier is behind every wave's last read, and a wave's copies are all done
    wgrad_wide_run<kOutF32>(aq, sa, bq, sb, offsets, G, M, all_tiles, P, Q, g, static_cast<int64_t>(p) * kWideRows,
                            static_cast<int64_t>(q) * kTile, c, (FP8Q_LDS uint8_t *)stages);
  }
}

hipError_t launch_grouped_gemm_rowscaled(const uint8_t *aq, const float *sa, const uint8_t *bq, const float *sb,
                                         const int32_t *offsets, int64_t G, int64_t M, int64_t P, int64_t Q,
                                         void *c, bool out_f32, hipStream_t stream) {
  const int64_t cus = device_cu_count(), tp = P / kTile, tq = Q / kTile, tile = kTile * G;
  // Wide tiles for experts of 8 token tiles or more on average, with FP32 output 12, if that makes one for
  // every CU.  4 experts of 7168 x 2048 with 4, 8 and 12 token tiles, BF16: 60, 88 and 113 us by wide tiles,
  // 57, 92 and 125 by the others; with 12, FP32: 194 and 200; 32 of 4096 x 7168 with 8 and 12, FP32: 2380
  // and 3210 us, 2195 and 3125.  One expert of 2048 x 2048, half as many wide tiles as CUs, with 32:
  // BF16 29 and 30, FP32 53 and 46.  P = 128 would leave half of each wide tile empty (16 experts of
  // 128 x 8192 with 32 token tiles, BF16, 166 and 111 us).
  // M only bounds the rows, and how many are routed is known on the device: the value sort's default
  // capacity has room for every expert to be local.  So where M allows wide tiles both kernels are
  // launched, and the one that the offsets do not call for leaves at once (about 5 us).  8192 tokens x 8
  // slots, 32 of 256 experts of 4096 x 7168 local, 8192 of 65536 rows routed: FP32 1060 -> 850 us, BF16
  // 680 -> 510 against wide tiles by M.
  const int64_t wide = (P + kWideRows - 1) / kWideRows * tq;
  const int deepest = out_f32 ? 12 : 8;
  const bool maybe_wide = M >= deepest * tile && P > kTile && G * wide >= cus;
  // Tiles that a workgroup computes one after the other in a row of them: with few tokens per expert the
  // start of a workgroup (its expert's offsets, the first copies) costs as much as a tile.  Four, or two
  // for experts of half a token tile, as long as four workgroups per slot (two on a CU) remain.  32
  // experts of 7168 x 2048, BF16, by 1, 2, 4 and 8 tiles: 32 rows each 202, 151, 171 and 176 us, 128 rows
  // 243, 188, 180 and 177, 256 rows 306, 256, 251 and 245, 600 rows 476, 444, 427 and 458; FP32 less, 256
  // rows 453, 433, 413 and 419.
  int64_t run = G * tp * tq / (8 * cus);
  const int64_t longest = M < tile / 2 ? 2 : 4;
  run = run < 1 ? 1 : (run > longest ? longest : run);
  run = run > tq ? tq : run;
  auto small = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(8 * G * ((tp * ((tq + run - 1) / run) + 7) / 8))),
                       dim3(64 * kWaves), 0, stream, aq, sa, bq, sb, offsets, static_cast<int>(G), M, M / kTile + G,
                       static_cast<int>(P), static_cast<int>(Q), static_cast<int>(run), maybe_wide ? deepest : 0, c);
  };
  out_f32 ? small(wgrad_kernel<true>) : small(wgrad_kernel<false>);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !maybe_wide) return e;
  const int64_t units = 8 * G * ((wide + 7) / 8);
  auto large = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(units < 4 * cus ? units : 4 * cus)), dim3(64 * kWaves), 0, stream,
                       aq, sa, bq, sb, offsets, static_cast<int>(G), M, M / kTile + G, static_cast<int>(P),
                       static_cast<int>(Q), deepest, c);
  };
  out_f32 ? large(wgrad_wide_kernel<true>) : large(wgrad_wide_kernel<false>);
  return hipGetLastError();
}

}  // namespace fp8q
