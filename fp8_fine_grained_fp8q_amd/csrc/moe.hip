// Expert-parallel dispatch and combine around the grouped GEMM, one GPU's share, for gfx950.
//
// Each token is routed to 8 of 256 experts (dlbhg.com page on DeepSeek-V3's training
// techniques, section 1.1, item 2), the experts are spread over the GPUs (same page, section
// 2.1: 64-way expert parallelism) and tokens reach their experts and come back by all-to-all
// dispatch and combine (same page, section 3.1; dtcms.com page, the DualPipe paragraph).
// The exchange itself needs several GPUs; these kernels are the work on either side of it
// on the GPU that owns experts [e_begin, e_begin + E):
//   * route: from the top-k expert ids of T tokens, the expert-sorted row of every (token,
//     slot) routed to a local expert (experts in order, tokens ascending within one), the
//     per-expert offsets the grouped GEMM reads, and the inverse map for the combine;
//   * pack: copy each such row's E4M3 codes and 1x128 tile scales into that layout (the
//     activation quantizer is row-local, so quantizing before the exchange is the same as
//     after it, and the payload is the FP8 codes plus 4 bytes per 128 of them);
//   * combine: y[t] = sum over the token's local slots s of w[t, s] * out[row(t, s)], FP32
//     accumulation in slot order.
//   * sort: the same route with BF16 or FP32 rows in place of codes (the weight gradient
//     quantizes them along the tokens), and the gradients of the sort and of the combine.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kMaxLocalExperts = 1024;
constexpr int64_t kAloneChunks = 16;  // up to here a routing is one launch (launch_route)
constexpr int64_t kChunk = 1024;  // (token, slot) entries per routing workgroup; >= kMaxLocalExperts

// Count of the set bits of mask below this lane.
__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return static_cast<int>(__builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                                    __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0u)));
}

// The routing splits the n = T*k entries into C = max(1, floor(n / kChunk)) chunks of
// kChunk entries in order, the last one taking the remainder (so every chunk but a lone one
// holds at least kChunk >= E entries).  Entry range of chunk c:
__device__ __forceinline__ void chunk_range(int64_t c, int64_t C, int64_t n, int64_t &lo, int64_t &hi) {
  lo = c * kChunk;
  hi = c == C - 1 ? n : lo + kChunk;
}

__device__ __forceinline__ int local_expert(const int32_t *__restrict__ ids, int64_t idx, int64_t hi,
                                            int64_t e_begin, int E) {
  if (idx >= hi) return -1;
  const int64_t g = static_cast<int64_t>(ids[idx]) - e_begin;
  return g >= 0 && g < E ? static_cast<int>(g) : -1;
}

// Exclusive prefix sum of v over the kRouteThreads threads in thread order; *total gets the
// sum.  Every thread of the workgroup calls it; ws is kRouteWaves ints of LDS.
__device__ __forceinline__ int block_exclusive_scan(int v, int *ws, int *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(inc, d);
    if (lane >= d) inc += u;
  }
  if (lane == 63) ws[wave] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRouteWaves; ++w) {
    const int t = ws[w];
    before += w < wave ? t : 0;
    all += t;
  }
  __syncthreads();  // ws may be reused after this
  *total = all;
  return before + inc - v;
}

// 1 (C > kAloneChunks only): each workgroup counts its chunk's entries per local expert and leaves the
// counts in the first E entries of its own range of token_row, which the ranking pass
// overwrites later (only this chunk's workgroups ever touch that range).
__global__ __launch_bounds__(kRouteThreads) void moe_count_kernel(const int32_t *__restrict__ ids, int64_t n,
                                                                  int64_t C, int64_t e_begin, int E,
                                                                  int32_t *__restrict__ token_row) {
  __shared__ int32_t hist[kMaxLocalExperts];
  int64_t lo, hi;
  chunk_range(blockIdx.x, C, n, lo, hi);
  for (int e = threadIdx.x; e < E; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
  for (int64_t i = lo + threadIdx.x; i < hi; i += kRouteThreads) {
    const int e = local_expert(ids, i, hi, e_begin, E);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kRouteThreads) token_row[lo + e] = hist[e];
}

// 2 (C > kAloneChunks only), one workgroup: offsets[e] = rows of the experts before e, and in place of
// chunk c's count of expert e, that chunk's first row of expert e (offsets[e] plus the counts
// of the earlier chunks).  Thread (g, e) = (tid / E, tid % E) walks a contiguous run of
// chunks for expert e; the runs' sums are scanned per expert, the experts' totals over the
// workgroup.
__global__ __launch_bounds__(kRouteThreads) void moe_scan_kernel(int64_t n, int64_t C, int E,
                                                                 int32_t *__restrict__ offsets,
                                                                 int32_t *__restrict__ token_row) {
  __shared__ int32_t part[kRouteThreads];
  __shared__ int32_t first[kMaxLocalExperts];
  __shared__ int32_t ws[kRouteWaves];
  const int tid = threadIdx.x;
  const int G = kRouteThreads / E;
  const int64_t per = (C + G - 1) / G;
  const int g = tid / E, e = tid % E;
  const int64_t c_lo = g < G ? g * per : C, c_hi = c_lo + per < C ? c_lo + per : C;
  int s = 0;
#pragma unroll 8
  for (int64_t c = c_lo; c < c_hi; ++c) s += token_row[c * kChunk + e];  // independent loads
  if (g < G) part[tid] = s;
  __syncthreads();
  int tot = 0;
  if (tid < E) {
    for (int j = 0; j < G; ++j) {  // runs before g, per expert
      const int p = part[j * E + tid];
      part[j * E + tid] = tot;
      tot += p;
    }
  }
  int all;
  const int ex = block_exclusive_scan(tid < E ? tot : 0, ws, &all);
  if (tid < E) {
    offsets[tid] = ex;
    first[tid] = ex;
  }
  if (tid == 0) offsets[E] = all;
  __syncthreads();
  int base = g < G ? first[e] + part[tid] : 0;
#pragma unroll 8
  for (int64_t c = c_lo; c < c_hi; ++c) {
    const int v = token_row[c * kChunk + e];
    token_row[c * kChunk + e] = base;
    base += v;
  }
}

// Adds the local experts' counts of the entries [lo, hi) to hist (LDS, any number of waves).  The
// lanes that share the first local lane's expert are added at once, so that a batch routed
// mostly to one expert does not queue up at its counter.
__device__ __forceinline__ void count_entries(const int32_t *__restrict__ ids, int64_t lo, int64_t hi, int64_t e_begin,
                                              int E, int32_t *hist) {
  const int lane = threadIdx.x & 63;
  constexpr int U = 4;  // entries per thread in flight
  for (int64_t i0 = lo; i0 < hi; i0 += U * kRouteThreads) {
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) e[u] = local_expert(ids, i0 + u * kRouteThreads + threadIdx.x, hi, e_begin, E);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint64_t here = __ballot(e[u] >= 0);
      if (here == 0) continue;
      const int first = __ffsll(static_cast<unsigned long long>(here)) - 1;
      const int common = __builtin_amdgcn_readlane(e[u], first);
      const uint64_t same = __ballot(e[u] == common);
      if (lane == first)
        atomicAdd(&hist[common], __popcll(same));
      else if (e[u] >= 0 && e[u] != common)
        atomicAdd(&hist[e[u]], 1);
    }
  }
}

// 3: each workgroup ranks its chunk, 1024 entries per round, one per thread.  Within a wave
// the lanes of one expert are found without a loop: the ballots of the expert index's bits
// (and of "local") intersect to the set of lanes with this lane's expert.  A lane's row is
// the chunk's running row of its expert, plus that expert's entries in the earlier waves of
// the round, plus those in lower lanes, so rows follow entry order, i.e. token order within
// an expert.  With few chunks (kAlone; a lone one among them) the passes before are not run: each
// workgroup counts all entries by itself, those before its chunk first, and scans the counts; the
// first one writes the offsets.
template <bool kAlone>
__global__ __launch_bounds__(kRouteThreads) void moe_rank_kernel(const int32_t *__restrict__ ids, int64_t n,
                                                                 int64_t C, int k, int64_t e_begin, int E,
                                                                 int64_t cap, int32_t *__restrict__ offsets,
                                                                 int32_t *__restrict__ token_row,
                                                                 int32_t *__restrict__ row_token) {
  __shared__ int32_t run[kMaxLocalExperts];                  // the chunk's next row, per expert
  __shared__ int32_t wcnt[kRouteWaves * kMaxLocalExperts];   // a round's count per wave and expert
  __shared__ int32_t ws[kRouteWaves];
  const int tid = threadIdx.x, wave = tid >> 6;
  int64_t lo, hi;
  chunk_range(blockIdx.x, C, n, lo, hi);
  for (int i = tid; i < kRouteWaves * E; i += kRouteThreads) wcnt[i] = 0;
  if (!kAlone) {
    for (int e = tid; e < E; e += kRouteThreads) run[e] = token_row[lo + e];
  } else {
    for (int e = tid; e < E; e += kRouteThreads) run[e] = 0;
    __syncthreads();
    count_entries(ids, 0, lo, e_begin, E, run);
    __syncthreads();
    const int earlier = tid < E ? run[tid] : 0;
    __syncthreads();
    count_entries(ids, lo, n, e_begin, E, run);
    __syncthreads();
    int all;
    const int cnt = tid < E ? run[tid] : 0;
    const int ex = block_exclusive_scan(cnt, ws, &all);
    if (tid < E) {
      run[tid] = ex + earlier;
      if (blockIdx.x == 0) offsets[tid] = ex;
    }
    if (blockIdx.x == 0 && tid == 0) offsets[E] = all;
  }
  __syncthreads();  // the counts in token_row are read before this chunk's rows overwrite them
  const int nbits = E > 1 ? 32 - __clz(E - 1) : 0;
  for (int64_t r0 = lo; r0 < hi; r0 += kRouteThreads) {
    const int64_t idx = r0 + tid;
    const int e = local_expert(ids, idx, hi, e_begin, E);
    uint64_t m = __ballot(e >= 0);
    for (int b = 0; b < nbits; ++b) {
      const uint64_t bit = __ballot(e >= 0 && ((e >> b) & 1));
      m &= ((e >> b) & 1) ? bit : ~bit;
    }
    const bool leader = e >= 0 && lanes_below(m) == 0;
    if (leader) wcnt[wave * E + e] = __popcll(m);
    __syncthreads();
    int row = -1, last_wave = -1, round_total = 0;
    if (e >= 0) {
      int before = 0;
#pragma unroll
      for (int w = 0; w < kRouteWaves; ++w) {
        const int t = wcnt[w * E + e];
        before += w < wave ? t : 0;
        round_total += t;
        last_wave = t > 0 ? w : last_wave;
      }
      row = run[e] + before + lanes_below(m);
    }
    __syncthreads();  // every lane has read run[] and wcnt[]
    if (leader) {
      wcnt[wave * E + e] = 0;
      if (last_wave == wave) run[e] += round_total;
    }
    // rows past the capacity are dropped (their slots read as not local); offsets still count
    // them, so the caller can see that the capacity was too small
    if (idx < hi) token_row[idx] = row < cap ? row : -1;
    if (row >= 0 && row < cap) row_token[row] = static_cast<int32_t>(idx / k);
    __syncthreads();
  }
}

// One wave per dispatched row r < offsets[E]: the token's K code bytes (16 per lane and
// step) and its K/128 tile scales (sa[kb][t] -> sa_s[kb][r], row stride `cap`).
__global__ __launch_bounds__(256) void moe_pack_kernel(const uint8_t *__restrict__ xq, const float *__restrict__ sa,
                                                       int64_t T, int64_t K, const int32_t *__restrict__ row_token,
                                                       const int32_t *__restrict__ offsets, int E, int64_t cap,
                                                       uint8_t *__restrict__ xq_s, float *__restrict__ sa_s) {
  const int lane = threadIdx.x & 63;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (r >= offsets[E] || r >= cap) return;
  const int64_t t = row_token[r];
  const uint4 *src = reinterpret_cast<const uint4 *>(xq + t * K);
  uint4 *dst = reinterpret_cast<uint4 *>(xq_s + r * K);
  for (int64_t i = lane; i < K / 16; i += 64) dst[i] = src[i];
  for (int64_t kb = lane; kb < K / 128; kb += 64) sa_s[kb * cap + r] = sa[kb * T + t];
}

// One workgroup per token; each thread takes 8 consecutive columns at a time.  The slots
// are visited in order and each adds w * out[row] with one FMA per element.
template <bool kInF32, bool kOutF32>
__global__ __launch_bounds__(256) void moe_combine_kernel(const void *__restrict__ out, int64_t N,
                                                          const int32_t *__restrict__ token_row,
                                                          const float *__restrict__ w, int k, int64_t cap,
                                                          void *__restrict__ y) {
  const int64_t t = blockIdx.x;
  for (int64_t c = threadIdx.x; c < N / 8; c += 256) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < k; ++s) {
      const int32_t r = token_row[t * k + s];
      if (r < 0 || r >= cap) continue;  // not a local slot (or not a row of `out`)
      const float ws = w[t * k + s];
      float v[8];
      load8<kInF32>(out, static_cast<int64_t>(r) * N + 8 * c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(ws, v[i], acc[i]);
    }
    if (kOutF32) {
      float *yo = static_cast<float *>(y) + t * N + 8 * c;
      *reinterpret_cast<float4 *>(yo) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      *reinterpret_cast<float4 *>(yo + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else {
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(acc[i]);
        b[i] = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;  // round to nearest even
      }
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(y) + t * N + 8 * c) =
          make_uint4(b[0] | (b[1] << 16), b[2] | (b[3] << 16), b[4] | (b[5] << 16), b[6] | (b[7] << 16));
    }
  }
}

// The rows of token t, one per lane: lane s < k holds token_row[t][s] if that is a row of the
// sorted layout (0 <= row < cap); the set of such lanes is returned.  One coalesced load
// serves all k slots, and the loops below run over the slots that have a row only.
__device__ __forceinline__ uint64_t token_rows(const int32_t *__restrict__ token_row, int64_t t, int k, int64_t cap,
                                               int32_t &row) {
  const int lane = threadIdx.x & 63;
  row = lane < k ? token_row[t * k + lane] : -1;
  return __ballot(row >= 0 && row < cap);
}

// Sorted rows (the values a weight gradient needs, where the dispatch carries codes):
// xs[token_row[t][s]] = x[t].  Driven by the tokens, so that each token's row is read once
// however many local experts it has; a workgroup takes 256 U 16-byte chunks of one token.
template <int U>
__global__ __launch_bounds__(256) void moe_spread_kernel(const u32x4 *__restrict__ x, int64_t chunks, int segs,
                                                         const int32_t *__restrict__ token_row, int k, int64_t cap,
                                                         u32x4 *__restrict__ xs) {
  const int64_t t = blockIdx.x / segs;
  const int64_t c = static_cast<int64_t>(blockIdx.x % segs) * (256 * U) + threadIdx.x;
  int32_t row;
  uint64_t todo = token_rows(token_row, t, k, cap, row);
  if (todo == 0) return;
  u32x4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c + 256 * u < chunks) v[u] = x[t * chunks + c + 256 * u];
  for (; todo != 0; todo &= todo - 1) {
    const int64_t r = __builtin_amdgcn_readlane(row, __ffsll(static_cast<unsigned long long>(todo)) - 1);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + 256 * u < chunks) __builtin_nontemporal_store(v[u], xs + (r * chunks + c + 256 * u));
  }
}

// Gradient of the sort: dx[t] = sum over the token's slots with a row of dxs[row], FP32, in
// slot order, rounded once.  A workgroup takes 256 chunks of 8 columns of one token; up to four
// rows are read at once.
template <bool kInF32, bool kOutF32>
__global__ __launch_bounds__(256) void moe_sum_kernel(const void *__restrict__ dxs, int64_t H, int segs,
                                                      const int32_t *__restrict__ token_row, int k, int64_t cap,
                                                      void *__restrict__ dx) {
  const int64_t t = blockIdx.x / segs;
  // Threads past the row's end sum its first chunk and store nothing: no lane leaves before the
  // loop, which reads `row` from all of them.
  const int64_t own = static_cast<int64_t>(blockIdx.x % segs) * 256 + threadIdx.x;
  const bool in = own < H / 8;
  const int64_t c = in ? own : 0;
  int32_t row;
  uint64_t todo = token_rows(token_row, t, k, cap, row);
  auto next = [&]() -> int64_t {
    const int64_t r = __builtin_amdgcn_readlane(row, __ffsll(static_cast<unsigned long long>(todo)) - 1);
    todo &= todo - 1;
    return r * H + 8 * c;
  };
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto add = [&](auto batch) {
    constexpr int n = decltype(batch)::value;
    float v[n][8];
#pragma unroll
    for (int j = 0; j < n; ++j) load8<kInF32>(dxs, next(), v[j]);
#pragma unroll
    for (int j = 0; j < n; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[j][i];
  };
  while (__popcll(todo) >= 4) add(std::integral_constant<int, 4>{});
  if (__popcll(todo) >= 2) add(std::integral_constant<int, 2>{});
  if (todo != 0) add(std::integral_constant<int, 1>{});
  if (in) store8<kOutF32>(dx, t * H + 8 * c, acc);
}

// The whole sort of at most kSmallSort entries in one launch (a lone routing chunk: the routing
// kernel and the copy would be two).  Every workgroup holds all local expert indices in LDS and
// finds its token's rows by counting, row = the entries of an earlier expert, or of the same
// one and earlier in order: one ballot per 64 entries and slot.  The last workgroup counts the
// offsets.  64 tokens x 8 slots x 7168 BF16 columns: 2.7 us less a call than by two launches; the
// kernel takes 6.0.
constexpr int kSmallSort = 2 * static_cast<int>(kChunk) - 1;

__global__ __launch_bounds__(256) void moe_sort_small_kernel(const int32_t *__restrict__ ids, int n, int k,
                                                             int64_t e_begin, int E, const uint4 *__restrict__ x,
                                                             int64_t chunks, int segs, int64_t cap,
                                                             uint4 *__restrict__ xs, int32_t *__restrict__ offsets,
                                                             int32_t *__restrict__ token_row,
                                                             int32_t *__restrict__ row_token) {
  __shared__ int32_t key[kSmallSort + 1];  // local expert index, E where there is none
  __shared__ int32_t rows[64];
  __shared__ int32_t hist[kMaxLocalExperts + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < n; i += 256) {
    const int e = local_expert(ids, i, n, e_begin, E);
    key[i] = e < 0 ? E : e;
  }
  if (blockIdx.x == gridDim.x - 1) {  // offsets[e] = the entries of the experts before e
    for (int e = tid; e <= E; e += 256) hist[e] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += 256) atomicAdd(&hist[key[i]], 1);
    __syncthreads();
    if (wave != 0) return;
    int before = 0;
    for (int e0 = 0; e0 <= E; e0 += 64) {
      const int e = e0 + lane, own = e < E ? hist[e] : 0;
      int sum = own;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(sum, d);
        sum += lane >= d ? u : 0;
      }
      if (e <= E) offsets[e] = before + sum - own;
      before += __shfl(sum, 63);
    }
    return;
  }
  __syncthreads();
  const int t = blockIdx.x / segs, seg = blockIdx.x % segs;
  for (int s = wave; s < k; s += 4) {
    const int i = t * k + s, own = key[i];
    int row = 0;
    for (int j0 = 0; own < E && j0 < n; j0 += 64) {
      const int j = j0 + lane, e = j < n ? key[j] : E;
      row += __popcll(__ballot(e < own || (e == own && j < i)));
    }
    if (own >= E || row >= cap) row = -1;
    if (lane == 0) {
      rows[s] = row;
      if (seg == 0) {
        token_row[i] = row;
        if (row >= 0) row_token[row] = t;
      }
    }
  }
  __syncthreads();
  const int64_t c = static_cast<int64_t>(seg) * 256 + tid;
  if (c >= chunks) return;
  const uint4 v = x[t * chunks + c];
  for (int s = 0; s < k; ++s) {
    const int64_t r = rows[s];
    if (r >= 0) xs[r * chunks + c] = v;
  }
}

// Gradient of the combine, one wave per (token, slot): dout[row] = w * dy[t] in the expert
// outputs' type and dw = <out[row], dy[t]>, FP32 (each lane sums its columns in order, then
// a fixed tree over the lanes: the same bits in every run).  A slot without a row gets
// dw = 0.  The waves of a token share a workgroup or sit in neighbouring ones, so dy comes
// from the caches after its first read.
template <bool kF32, bool kDyF32>
__global__ __launch_bounds__(256) void moe_combine_backward_kernel(const void *__restrict__ dy,
                                                                   const void *__restrict__ out, int64_t N,
                                                                   const int32_t *__restrict__ token_row,
                                                                   const float *__restrict__ w, int64_t n, int k,
                                                                   int64_t cap, void *__restrict__ dout,
                                                                   float *__restrict__ dw) {
  const int lane = threadIdx.x & 63;
  const int64_t entry = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (entry >= n) return;
  const int64_t r = token_row[entry];
  float sum = 0.0f;
  if (r >= 0 && r < cap) {
    const int64_t t = entry / k;
    const float ws = w[entry];
    for (int64_t c = lane; c < N / 8; c += 64) {
      float d[8], o[8];
      load8<kDyF32>(dy, t * N + 8 * c, d);
      load8<kF32>(out, r * N + 8 * c, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum = __builtin_fmaf(o[i], d[i], sum);
        d[i] *= ws;
      }
      store8<kF32>(dout, r * N + 8 * c, d);
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m);
  }
  if (lane == 0) dw[entry] = sum;
}

namespace {

// The routing launches shared by the dispatch and the sort: offsets, token_row, row_token.
hipError_t launch_route(const int32_t *ids, int64_t T, int64_t k, int64_t e_begin, int64_t E, int64_t cap,
                        int32_t *offsets, int32_t *token_row, int32_t *row_token, hipStream_t stream) {
  const int64_t n = T * k, C = n / kChunk > 1 ? n / kChunk : 1;
  if (E < 1 || E > kMaxLocalExperts || C > 0x7fffffff) return hipErrorInvalidValue;
  const int kk = static_cast<int>(k), EE = static_cast<int>(E);
  // Up to kAloneChunks chunks, one launch in which every chunk counts all entries; beyond, the
  // counts would cost more than the two launches that share them.  A sort call over 8 slots per token
  // and short rows: 2048 tokens (16 chunks) 14 against 20 us, 4096 19 against 20, 8192 30 against 19.
  if (C <= kAloneChunks) {
    hipLaunchKernelGGL(moe_rank_kernel<true>, dim3(static_cast<uint32_t>(C)), dim3(kRouteThreads), 0, stream, ids, n, C,
                       kk, e_begin, EE, cap, offsets, token_row, row_token);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(moe_count_kernel, dim3(static_cast<uint32_t>(C)), dim3(kRouteThreads), 0, stream, ids, n, C, e_begin,
                     EE, token_row);
  hipLaunchKernelGGL(moe_scan_kernel, dim3(1), dim3(kRouteThreads), 0, stream, n, C, EE, offsets, token_row);
  hipLaunchKernelGGL(moe_rank_kernel<false>, dim3(static_cast<uint32_t>(C)), dim3(kRouteThreads), 0, stream, ids, n, C, kk,
                     e_begin, EE, cap, offsets, token_row, row_token);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_dispatch(const int32_t *ids, int64_t T, int64_t k, int64_t e_begin, int64_t E,
                               const uint8_t *xq, const float *sa, int64_t K, int64_t cap, uint8_t *xq_s,
                               float *sa_s, int32_t *offsets, int32_t *token_row, int32_t *row_token,
                               hipStream_t stream) {
  if ((cap + 3) / 4 > 0x7fffffff) return hipErrorInvalidValue;
  hipError_t e = launch_route(ids, T, k, e_begin, E, cap, offsets, token_row, row_token, stream);
  if (e != hipSuccess || cap == 0) return e;
  hipLaunchKernelGGL(moe_pack_kernel, dim3(static_cast<uint32_t>((cap + 3) / 4)), dim3(256), 0, stream, xq, sa, T,
                     K, row_token, offsets, static_cast<int>(E), cap, xq_s, sa_s);
  return hipGetLastError();
}

namespace {

// 16-byte chunks of a row, and the workgroups that the copy takes for it.  Long rows: four chunks
// per thread, so that a workgroup's wait for its token's rows is paid once per row (8192 tokens x
// 7168, 32 of 256 experts local: 50.5 -> 45.5 us with the routing); shorter ones: a chunk per thread,
// more workgroups.
int64_t row_chunks(bool f32, int64_t H) { return H / (f32 ? 4 : 8); }
bool long_rows(int64_t chunks) { return chunks > 512; }
int64_t spread_segs(int64_t chunks) { return long_rows(chunks) ? (chunks + 1023) / 1024 : (chunks + 255) / 256; }

}  // namespace

int64_t moe_sort_groups(int64_t T, int64_t k, bool f32, int64_t H) {
  const int64_t chunks = row_chunks(f32, H);
  return T * k <= kSmallSort ? T * ((chunks + 255) / 256) + 1 : T * spread_segs(chunks);
}

hipError_t launch_moe_sort(const int32_t *ids, int64_t T, int64_t k, int64_t e_begin, int64_t E, const void *x,
                           bool f32, int64_t H, int64_t cap, void *xs, int32_t *offsets, int32_t *token_row,
                           int32_t *row_token, hipStream_t stream) {
  const int64_t chunks = row_chunks(f32, H), segs = (chunks + 255) / 256;
  if (E < 1 || E > kMaxLocalExperts) return hipErrorInvalidValue;
  if (T * k <= kSmallSort && segs > 0) {
    hipLaunchKernelGGL(moe_sort_small_kernel, dim3(static_cast<uint32_t>(T * segs + 1)), dim3(256), 0, stream, ids,
                       static_cast<int>(T * k), static_cast<int>(k), e_begin, static_cast<int>(E),
                       static_cast<const uint4 *>(x), chunks, static_cast<int>(segs), cap, static_cast<uint4 *>(xs),
                       offsets, token_row, row_token);
    return hipGetLastError();
  }
  hipError_t e = launch_route(ids, T, k, e_begin, E, cap, offsets, token_row, row_token, stream);
  if (e != hipSuccess || cap == 0 || T * segs == 0) return e;
  const int64_t per = spread_segs(chunks);
  auto spread = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(T * per)), dim3(256), 0, stream,
                       static_cast<const u32x4 *>(x), chunks, static_cast<int>(per), token_row, static_cast<int>(k), cap,
                       static_cast<u32x4 *>(xs));
  };
  long_rows(chunks) ? spread(moe_spread_kernel<4>) : spread(moe_spread_kernel<1>);
  return hipGetLastError();
}

hipError_t launch_moe_sort_backward(const void *dxs, bool in_f32, int64_t cap, int64_t H, const int32_t *token_row,
                                    int64_t T, int64_t k, void *dx, bool out_f32, hipStream_t stream) {
  const int64_t segs = (H / 8 + 255) / 256;
  const dim3 grid(static_cast<uint32_t>(T * segs)), block(256);
  const int kk = static_cast<int>(k);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, dxs, H, static_cast<int>(segs), token_row, kk, cap, dx); };
  if (in_f32)
    out_f32 ? go(moe_sum_kernel<true, true>) : go(moe_sum_kernel<true, false>);
  else
    out_f32 ? go(moe_sum_kernel<false, true>) : go(moe_sum_kernel<false, false>);
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void *dy, bool dy_f32, const void *out, bool f32, int64_t cap, int64_t N,
                                       const int32_t *token_row, const float *w, int64_t T, int64_t k, void *dout,
                                       float *dw, hipStream_t stream) {
  const int64_t n = T * k;
  const dim3 grid(static_cast<uint32_t>((n + 3) / 4)), block(256);
  const int kk = static_cast<int>(k);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, dy, out, N, token_row, w, n, kk, cap, dout, dw);
  };
  if (f32)
    dy_f32 ? go(moe_combine_backward_kernel<true, true>) : go(moe_combine_backward_kernel<true, false>);
  else
    dy_f32 ? go(moe_combine_backward_kernel<false, true>) : go(moe_combine_backward_kernel<false, false>);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void *out, bool in_f32, int64_t cap, int64_t N, const int32_t *token_row,
                              const float *w, int64_t T, int64_t k, void *y, bool out_f32, hipStream_t stream) {
  if (T > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>(T)), block(256);
  const int kk = static_cast<int>(k);
  if (in_f32 && out_f32)
    hipLaunchKernelGGL((moe_combine_kernel<true, true>), grid, block, 0, stream, out, N, token_row, w, kk, cap, y);
  else if (in_f32)
    hipLaunchKernelGGL((moe_combine_kernel<true, false>), grid, block, 0, stream, out, N, token_row, w, kk, cap, y);
  else if (out_f32)
    hipLaunchKernelGGL((moe_combine_kernel<false, true>), grid, block, 0, stream, out, N, token_row, w, kk, cap, y);
  else
    hipLaunchKernelGGL((moe_combine_kernel<false, false>), grid, block, 0, stream, out, N, token_row, w, kk, cap, y);
  return hipGetLastError();
}

}  // namespace fp8q
