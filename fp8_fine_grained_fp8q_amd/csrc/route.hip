// The router of an MoE layer: top-k experts per token with their gating weights, the counts per
// expert, the balance loss, and the gradient with respect to the logits, for gfx950.  The expert ids
// feed the dispatch and the sort, the weights the combine (dlbhg.com page on DeepSeek-V3's training
// techniques, section 1.1 item 2: 8 of 256 routed experts, a bias per expert that steers the
// selection only, and a small sequence-wise balance loss).
//
// Scores s of a token: softmax(z) or sigmoid(z) of its logits z.  Chosen are the k largest of
// s + bias (of z without a bias: both scores rise with z), ties to the lower index; an expert with
// logit -inf is never chosen.  Weights w_j = scale s_j (softmax, sigmoid), or normalized over the
// chosen ones, w_j = scale s_j / sum_i s_i.  With p = s / sum_e s_e, a sequence's counts c_e and its
// n tokens (valid ones with an expert), and B sequences,
//   slope_e = balance / B * E c_e / (n sum_e c_e),  loss = sum over sequences and e of slope_e sum_t p_te,
// so slope is the loss's derivative by every p_te of the sequence.  Backward, with g = dloss slope
// and d_j = dw_j w_j (normalized: w_j (dw_j - sum_i w_i dw_i / scale), a softmax over the chosen):
//   softmax:  dz_e = p_e (g_e - sum p g) + [e chosen] d_j, less p_e sum_i w_i dw_i if not normalized,
//   sigmoid:  dz_e = (1 - s_e) (p_e (g_e - sum p g) + [e chosen] d_j).
//
// The ranks are those of scores computed in 64 bits.  Scores in FP32 give the same ones unless two
// that follow each other are nearer than their errors; then the chosen ones and those beside the last of them are
// ranked by their 64-bit scores (about one token in 500 with sigmoid scores).
//
// Sigmoid scores of a token may all lie below FP32's range.  Normalized weights and shares p are therefore formed
// from scores times e^-m, with m the largest logit, of the chosen ones or of all, and at most 0.
//
// A group of 16 lanes takes a token of up to 256 experts, 64 lanes one of up to 1024, 4 to 16
// logits per lane in registers: the maxima of a top-k step are 4 DPP steps inside a row of lanes, and
// one instruction works for 4 tokens.  Logits are read once (16 MB for 16384 tokens x 256 experts,
// 3 us of HBM time).  What bounds the call is the time of one token: k maxima that follow each other over FP64 keys, the
// exponentials and the ways through LDS, 14.7 us for 64 tokens with sigmoid scores and a bias.  The
// instance for 256 experts takes 184 registers and 58 KB of LDS, one workgroup of 512 threads per CU, so that 16384 tokens in
// four sequences are 512 workgroups in two rounds of it: 31 us (fewer registers by launch bounds were slower).  512 and 1024
// experts, 16384 tokens: 90 and 94 us for the whole call.  With all 256 experts ranked in 64 bits for the tokens that
// FP32 leaves open it took 41.  Counts and sums of p stay in a workgroup's LDS and registers; a second launch
// (4 to 7 us) adds them up to slope and loss.
// The gradient reads and writes 33 MB in 14 us.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "fp8q.h"
#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

namespace {

constexpr int kRouteThreads = 512;  // the most of a workgroup
constexpr int kNoExpert = 0x7fffffff;

template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_amdgcn_update_dpp(0.0f, v, kCtrl, 0xf, 0xf, false);
}
template <int kCtrl>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, kCtrl, 0xf, 0xf, false);
}
template <int kCtrl>
__device__ __forceinline__ double dpp(double v) {
  const int64_t b = __builtin_bit_cast(int64_t, v);
  const uint32_t lo = dpp<kCtrl>(static_cast<int>(b)), hi = dpp<kCtrl>(static_cast<int>(b >> 32));
  return __builtin_bit_cast(double, static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo));
}

// op over the kLanes lanes (16 or 64) of a token, in every one of them.
template <int kLanes, class V, class Op>
__device__ __forceinline__ V across(V v, Op op) {
  v = op(v, dpp<0x128>(v));  // row_ror 8, 4, 2, 1
  v = op(v, dpp<0x124>(v));
  v = op(v, dpp<0x122>(v));
  v = op(v, dpp<0x121>(v));
  if (kLanes == 64) {
    v = op(v, __shfl_xor(v, 16));
    v = op(v, __shfl_xor(v, 32));
  }
  return v;
}

struct Add {
  template <class V>
  __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};
struct Min {
  __device__ __forceinline__ int operator()(int a, int b) const { return a < b ? a : b; }
};

// Lane `l`'s value v belongs to expert 4 (l + kLanes (v / 4)) + v % 4: four neighbours per load.
template <int kLanes>
__device__ __forceinline__ int expert_of(int l, int v) {
  return 4 * (l + kLanes * (v >> 2)) + (v & 3);
}

// The logits of one token in FP32, -inf past the last expert.
template <int kLanes, int kV, bool kF32>
__device__ __forceinline__ void load_logits(const void *p, int64_t row, int E, int l, float (&z)[kV]) {
  const int64_t at = row * E;
  if ((E & 3) == 0) {  // then every row is aligned for four values
#pragma unroll
    for (int j = 0; j < kV / 4; ++j) {
      const int e = 4 * (l + kLanes * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[4 * j + i] = -INFINITY;
      if (e < E) {
        if (kF32) {
          const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at + e);
          z[4 * j] = v.x, z[4 * j + 1] = v.y, z[4 * j + 2] = v.z, z[4 * j + 3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + at + e);
          z[4 * j] = bf16_lo(v.x), z[4 * j + 1] = bf16_hi(v.x), z[4 * j + 2] = bf16_lo(v.y), z[4 * j + 3] = bf16_hi(v.y);
        }
      }
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int e = expert_of<kLanes>(l, v);
    z[v] = -INFINITY;
    if (e < E) z[v] = kF32 ? static_cast<const float *>(p)[at + e] : bf16_lo(static_cast<const uint16_t *>(p)[at + e]);
  }
}

template <bool kF32>
__device__ __forceinline__ float load_logit(const void *p, int64_t at) {
  return kF32 ? static_cast<const float *>(p)[at] : bf16_lo(static_cast<const uint16_t *>(p)[at]);
}

// e^x for x <= 0, to 2^-22 of itself (0 below FP32's normal range): the hardware's 2^y at y = x log2 e rounded,
// times 1 + ln 2 of what y lost.  7 instructions instead of 20.
__device__ __forceinline__ float exp_of(float x) {
  x = fmaxf(x, -1000.0f);  // also -inf, whose loss would be NaN
  const float y = x * 1.44269502f;
  const float rest = __builtin_fmaf(x, 1.92596303e-8f, __builtin_fmaf(x, 1.44269502f, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return __builtin_fmaf(e, rest * 0.693147182f, e);
}

// 1 / x for x in [1, 2], to one unit of the last place.
__device__ __forceinline__ float reciprocal(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return __builtin_fmaf(r, __builtin_fmaf(-x, r, 1.0f), r);
}

// 1 / (1 + e^-z) and 1 minus it, from e^-|z|: no overflow, no cancellation.  -inf gives 0 and 1.
__device__ __forceinline__ float sigmoid(float z, float &rest) {
  const float t = exp_of(-fabsf(z)), r = reciprocal(1.0f + t);
  rest = (z >= 0.0f ? t : 1.0f) * r;
  return (z >= 0.0f ? 1.0f : t) * r;
}

// e^(z - top) or sigmoid(z) of a token's logits, their sum, and the logits' maximum.
template <int kLanes, int kV, bool kSoftmax>
__device__ __forceinline__ void scores(const float (&z)[kV], float (&s)[kV], float &sum, float &top) {
  top = z[0];
#pragma unroll
  for (int v = 1; v < kV; ++v) top = fmaxf(top, z[v]);
  top = across<kLanes>(top, Max{});
  sum = 0.0f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    float rest;
    s[v] = kSoftmax ? exp_of(z[v] - top) : sigmoid(z[v], rest);
    sum += s[v];
  }
  sum = across<kLanes>(sum, Add{});
}

// Sigmoid scores and their sum times e^-min(top, 0) in place of those of `scores`: tokens whose scores are all below FP32's
// range keep their shares p = s / sum s.  The same bits where top >= 0, and called only where a token of the wave has
// another one: a second exponential per logit.
template <int kLanes, int kV>
__device__ __forceinline__ void raise_scores(const float (&z)[kV], float top, float (&s)[kV], float &sum) {
  const float m = fminf(top, 0.0f);
  sum = 0.0f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    s[v] = exp_of(fminf(z[v], 0.0f) - m) * reciprocal(1.0f + exp_of(-fabsf(z[v])));
    sum += s[v];
  }
  sum = across<kLanes>(sum, Add{});
}

// LDS that one lane of a wave has written is read by another one behind this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Keys of the top-k with their expert, as one number that sorts by the key and then by the lower index: an FP32
// number as FP64 has 29 zero bits at its end, so that one maximum finds both.  Keys of -inf (and NaN) lie below kNone
// and are never chosen.
constexpr double kNone = -0x1p200, kLowest = -0x1p210;

__device__ __forceinline__ double pack(float key, int expert) {
  const double d = key > -INFINITY ? static_cast<double>(key + 0.0f) : kLowest;  // -0 as 0
  const int64_t bits = __builtin_bit_cast(int64_t, d);
  return __builtin_bit_cast(double, bits | static_cast<int64_t>(bits < 0 ? expert : 1023 - expert));
}

__device__ __forceinline__ int expert_in(double packed) {
  const int low = static_cast<int>(__builtin_bit_cast(int64_t, packed)) & 1023;
  return packed < 0.0 ? low : 1023 - low;
}

constexpr int kCandidates = 128;  // of a token whose order FP32 leaves open

// The largest packed key of a token, which is taken out.
template <int kLanes, int kV>
__device__ __forceinline__ double take_top(double (&key)[kV]) {
  double top = key[0];
#pragma unroll
  for (int v = 1; v < kV; ++v) top = fmax(top, key[v]);
  top = across<kLanes>(top, Max{});
#pragma unroll
  for (int v = 0; v < kV; ++v) key[v] = key[v] == top ? kLowest : key[v];
  return top;
}

// Top-k of packed keys (consumed): chosen expert j goes to ids[j] (LDS, one writer per token), -1 where no key
// is left.  With near > 0 also: every expert behind the k-th whose key differs from its by less than `near` times
// (its size + floor) follows there, `found` counts all of them, up to kCandidates + 1, and the answer
// is whether two keys that follow each other are as near.
template <int kLanes, int kV>
__device__ __forceinline__ bool select(double (&key)[kV], int k, int l, int32_t *ids, float near, float floor, int &found) {
  bool close = false;
  double last = 0.0;
  auto within = [&](double top) {
    return last - top <= static_cast<double>(near) * (fabs(last) + static_cast<double>(floor));
  };
  found = 0;
  for (int j = 0; j < k; ++j) {
    const double top = take_top<kLanes>(key);
    const bool some = top > kNone;
    if (l == 0) ids[j] = some ? expert_in(top) : -1;
    close |= near > 0.0f && j > 0 && some && within(top);
    found += some ? 1 : 0;
    last = top;
  }
  if (near > 0.0f) {
    bool more = found == k;
    while (true) {
      const double top = take_top<kLanes>(key);
      more = more && top > kNone && within(top) && found <= kCandidates;
      if (!__any(more)) break;
      if (more) {
        close = true;
        if (l == 0 && found < kCandidates) ids[found] = expert_in(top);
        ++found;
      }
    }
  }
  return close;
}

// A token's score + bias in 64 bits.
template <bool kSoftmax>
__device__ __forceinline__ double exact_score(double z, double top, double total, double bias) {
  return (kSoftmax ? exp(z - top) / total : 1.0 / (1.0 + exp(-z))) + bias;
}

// What a workgroup leaves in the workspace: FP32 sums of p [E], counts [E], its tokens and its routed
// slots.  In front of all of them a counter and the column blocks' parts of the loss.
constexpr int kColumns = 64;  // of a workgroup of the second kernel
constexpr int64_t kHead = 16;

int64_t column_blocks(int64_t E) { return (E + kColumns - 1) / kColumns; }

__device__ __forceinline__ float slope_of(double balance, int64_t B, int E, int count, int64_t routed, int64_t tokens) {
  const double n = static_cast<double>(routed) * static_cast<double>(tokens);
  return n > 0 ? static_cast<float>(balance / static_cast<double>(B) * E * count / n) : 0.0f;
}

struct RouteArgs {
  const void *logits;
  const float *bias;
  const uint8_t *valid;
  int32_t *ids;
  float *w;
  int32_t *counts;
  float *loss, *slope;
  uint32_t *counter;
  double *losses;
  float *parts;
  int64_t B, S;
  int E, k;
  bool normalize;
  float scale;
  double balance;
};

// Workgroup (x, y): tokens of sequence y, as many at a time as it has groups of kLanes lanes.  The
// only workgroup of a call writes the loss itself.
template <int kLanes, int kV, bool kSoftmax, bool kF32>
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(const RouteArgs a) {
  constexpr int kMost = kLanes * kV;                    // experts
  constexpr int kSlots = kMaxTopK / kLanes;        // of a lane
  __shared__ float sums[kRouteThreads / 64][kMost];
  __shared__ int32_t hist[kMost];
  __shared__ int32_t chosen[kRouteThreads / kLanes][kCandidates];
  __shared__ double exact[kRouteThreads / kLanes][kCandidates];
  __shared__ int32_t totals[2];
  __shared__ double loss[kRouteThreads / 64];
  const int l = threadIdx.x % kLanes, group = threadIdx.x / kLanes, groups = blockDim.x / kLanes;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int E = a.E, k = a.k;
  for (int e = threadIdx.x; e < kMost; e += blockDim.x) hist[e] = 0;
  if (threadIdx.x < 2) totals[threadIdx.x] = 0;
  __syncthreads();

  float bias[kV], far = 0.0f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int e = expert_of<kLanes>(l, v);
    bias[v] = a.bias != nullptr && e < E ? a.bias[e] : 0.0f;
    far = fmaxf(far, fabsf(bias[v]));
  }
  far = across<kLanes>(far, Max{});
  float sum_p[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) sum_p[v] = 0.0f;
  int tokens = 0, routed = 0;

  const int64_t stride = static_cast<int64_t>(gridDim.x) * groups;
  int32_t *const ids = chosen[group];
  // All lanes of a wave stay together: a group past the end works on logits of -inf.
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * groups; first < a.S; first += stride) {
    const int64_t t = first + group, row = blockIdx.y * a.S + t;
    bool here = t < a.S && (a.valid == nullptr || a.valid[row] != 0);
    float z[kV], s[kV], sum, top;
#pragma unroll
    for (int v = 0; v < kV; ++v) z[v] = -INFINITY;
    if (here) load_logits<kLanes, kV, kF32>(a.logits, row, E, l, z);
    scores<kLanes, kV, kSoftmax>(z, s, sum, top);
    here = here && top > -INFINITY;
    float r = 1.0f / sum;
    {
      double key[kV];
#pragma unroll
      for (int v = 0; v < kV; ++v)
        key[v] = pack(a.bias == nullptr || z[v] == -INFINITY ? z[v] : (kSoftmax ? s[v] * r : s[v]) + bias[v],
                      expert_of<kLanes>(l, v));
      if constexpr (!kSoftmax)  // the keys are packed: from here on s is for the shares
        if (__any(here && top < 0.0f)) {
          raise_scores<kLanes, kV>(z, top, s, sum);
          r = 1.0f / sum;
        }
      // A sigmoid in FP32 is off by less than 2^-21.5 of itself, a softmax by 2^-24 (12 + |z - top|), their sums with
      // the bias by 2^-24: 2^-19 and 2^-17 cover two of them, the latter down to scores of e^-50, and the
      // floor covers the smaller ones.  Scores end at 1, so a far larger bias (an expert's mask) adds nothing to it.
      const float near = a.bias == nullptr ? 0.0f : (kSoftmax ? 0x1p-17f : 0x1p-19f);
      int found;
      const bool close = select<kLanes, kV>(key, k, l, ids, near, fminf(2.0f * far + 1e-16f, 2.0f), found);
      if (__any(close)) {
        wave_sync();
        double total = 1.0;
        const double high = top;
        if (kSoftmax) {
          total = 0.0;
#pragma unroll 1
          for (int v = 0; v < kV; ++v) {
            const int e = expert_of<kLanes>(l, v);
            if (here && e < E) total += exp(static_cast<double>(load_logit<kF32>(a.logits, row * E + e)) - high);
          }
          total = across<kLanes>(total, Add{});
        }
        auto score_of = [&](int e) {
          return exact_score<kSoftmax>(load_logit<kF32>(a.logits, row * E + e), high, total, a.bias[e]);
        };
        if (close && found <= kCandidates) {
          // every candidate's place among them: those with a higher score, or as high and a lower index
          double *const score = exact[group];
#pragma unroll 1
          for (int c = l; c < found; c += kLanes) score[c] = score_of(ids[c]);
          wave_sync();
          int place[kCandidates / kLanes], id[kCandidates / kLanes];
#pragma unroll
          for (int i = 0; i < kCandidates / kLanes; ++i) {
            place[i] = k;
            id[i] = -1;
          }
#pragma unroll
          for (int i = 0; i < kCandidates / kLanes; ++i) {
            const int c = l + i * kLanes;
            if (c >= found) break;
            id[i] = ids[c];
            const double mine = score[c];
            int before = 0;
            for (int o = 0; o < found; ++o) before += score[o] > mine || (score[o] == mine && ids[o] < id[i]) ? 1 : 0;
            place[i] = before;
          }
          wave_sync();
#pragma unroll
          for (int i = 0; i < kCandidates / kLanes; ++i)
            if (place[i] < k) ids[place[i]] = id[i];
        } else if (close) {
          // more than that lie together (equal logits and biases): each rank by all scores
          uint32_t taken = 0;
#pragma unroll 1
          for (int j = 0; j < k; ++j) {
            double best = -INFINITY;
            int at = kNoExpert, v_at = 0;
#pragma unroll 1
            for (int v = 0; v < kV; ++v) {
              const int e = expert_of<kLanes>(l, v);
              if (e >= E || (taken >> v & 1u) != 0 || load_logit<kF32>(a.logits, row * E + e) == -INFINITY) continue;
              const double one = score_of(e);
              if (one > best) {
                best = one;
                at = e;
                v_at = v;
              }
            }
            const double most = across<kLanes>(best, Max{});
            const int won = across<kLanes>(best == most ? at : kNoExpert, Min{});
            if (won == at && at != kNoExpert) taken |= 1u << v_at;
            if (l == 0) ids[j] = won == kNoExpert ? -1 : won;
          }
        }
      }
    }
    wave_sync();
    here = here && ids[0] >= 0;  // without an expert (the bias masks those that the logits leave) a token counts for nothing
    if (here) {
      if (l == 0) ++tokens;
#pragma unroll
      for (int v = 0; v < kV; ++v) sum_p[v] += s[v] * r;
    }
    // Weights: slot j by lane j % kLanes.  Normalized ones are formed from scores times e^-m, with m
    // the largest chosen logit (sigmoid: at most 0), so that they do not vanish together.
    float x[kSlots], m = -INFINITY, total = 0.0f;
    int id[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int j = l + i * kLanes;
      id[i] = -1;
      if (i * kLanes >= k) break;
      id[i] = j < k && here ? ids[j] : -1;
      x[i] = id[i] >= 0 ? load_logit<kF32>(a.logits, row * E + id[i]) : -INFINITY;
      m = fmaxf(m, x[i]);
    }
    if (a.normalize) {
      m = across<kLanes>(m, Max{});
      if (!kSoftmax) m = fminf(m, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      if (i * kLanes >= k) break;
      float rest;
      if (a.normalize)
        x[i] = kSoftmax ? exp_of(x[i] - m) : exp_of(fminf(x[i], 0.0f) - m) * reciprocal(1.0f + exp_of(-fabsf(x[i])));
      else
        x[i] = kSoftmax ? exp_of(x[i] - top) * r : sigmoid(x[i], rest);
      total += id[i] >= 0 ? x[i] : 0.0f;
    }
    if (a.normalize) total = across<kLanes>(total, Add{});
    const float by = a.normalize ? a.scale / total : a.scale;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int j = l + i * kLanes;
      if (j >= k || t >= a.S) break;
      a.ids[row * k + j] = id[i];
      a.w[row * k + j] = id[i] >= 0 ? x[i] * by : 0.0f;
      if (id[i] >= 0) {
        ++routed;
        atomicAdd(&hist[id[i]], 1);
      }
    }
    wave_sync();  // ids is read before the next tokens' are written
  }

  // The workgroup's sums: of the groups of a wave, then of the waves, in this order.
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    if (kLanes == 16) {
      sum_p[v] += __shfl_xor(sum_p[v], 16);
      sum_p[v] += __shfl_xor(sum_p[v], 32);
    }
    if (lane < kLanes) sums[wave][expert_of<kLanes>(l, v)] = sum_p[v];
  }
  if (tokens) atomicAdd(&totals[0], tokens);
  if (routed) atomicAdd(&totals[1], routed);
  __syncthreads();
  const bool alone = gridDim.x == 1 && gridDim.y == 1;
  float *const part = a.parts + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * (2 * E + 2);
  double mine = 0.0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float p = 0.0f;
    for (int i = 0; i < waves; ++i) p += sums[i][e];
    if (alone) {
      const float slope = slope_of(a.balance, a.B, E, hist[e], totals[1], totals[0]);
      a.counts[e] = hist[e];
      a.slope[e] = slope;
      mine += static_cast<double>(slope) * static_cast<double>(p);
    } else {
      part[e] = p;
      part[E + e] = __int_as_float(hist[e]);
    }
  }
  if (!alone) {
    if (threadIdx.x < 2) part[2 * E + threadIdx.x] = __int_as_float(totals[threadIdx.x]);
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) *a.counter = 0;
    return;
  }
  for (int d = 32; d > 0; d >>= 1) mine += __shfl_xor(mine, d);
  if (lane == 0) loss[wave] = mine;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < waves; ++i) mine += loss[i];
  *a.loss = static_cast<float>(mine);
}

// Workgroup (x, y): 64 experts of sequence y from the sums of its `groups` workgroups, by 16 slices of
// them.  The last one to arrive adds up the parts of the loss, in order.
__global__ __launch_bounds__(1024) void moe_route_sum_kernel(const RouteArgs a, int groups) {
  __shared__ float p_of[16][kColumns];
  __shared__ int32_t count_of[16][kColumns];
  __shared__ int32_t totals[2][16];
  __shared__ bool last;
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6, E = a.E;
  const int e = blockIdx.x * kColumns + lane;
  const int64_t each = 2 * E + 2;
  const float *const part = a.parts + static_cast<int64_t>(blockIdx.y) * groups * each;
  float p = 0.0f;
  int count = 0, tokens = 0, routed = 0;
#pragma unroll 4
  for (int g = slice; g < groups; g += 16) {
    if (e < E) {
      p += part[g * each + e];
      count += __float_as_int(part[g * each + E + e]);
    }
    tokens += __float_as_int(part[g * each + 2 * E]);
    routed += __float_as_int(part[g * each + 2 * E + 1]);
  }
  p_of[slice][lane] = p;
  count_of[slice][lane] = count;
  if (lane == 0) {
    totals[0][slice] = tokens;
    totals[1][slice] = routed;
  }
  __syncthreads();
  if (slice != 0) return;
  tokens = 0;
  routed = 0;
  p = 0.0f;
  count = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    p += p_of[i][lane];
    count += count_of[i][lane];
    tokens += totals[0][i];
    routed += totals[1][i];
  }
  double mine = 0.0;
  if (e < E) {
    const int64_t at = static_cast<int64_t>(blockIdx.y) * E + e;
    const float slope = slope_of(a.balance, a.B, E, count, routed, tokens);
    a.counts[at] = count;
    a.slope[at] = slope;
    mine = static_cast<double>(slope) * static_cast<double>(p);
  }
  for (int d = 32; d > 0; d >>= 1) mine += __shfl_xor(mine, d);
  const uint32_t blocks = gridDim.x * gridDim.y;
  if (lane == 0) {
    __hip_atomic_store(&a.losses[blockIdx.y * gridDim.x + blockIdx.x], mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // the part of the loss has arrived; as an atomic of the device's scope it needs no fence, which would write
    // back the XCD's L2
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint32_t arrived = __hip_atomic_fetch_add(a.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = arrived + 1 == blocks;
  }
  wave_sync();
  if (!last) return;
  mine = 0.0;
  for (uint32_t i = lane; i < blocks; i += 64)
    mine += __hip_atomic_load(&a.losses[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int d = 32; d > 0; d >>= 1) mine += __shfl_xor(mine, d);
  if (lane == 0) *a.loss = static_cast<float>(mine);
}

struct RouteBackwardArgs {
  const void *logits;
  const int32_t *ids;
  const float *w, *dw, *slope, *dloss;
  void *dlogits;
  int64_t S;
  int E, k;
  bool normalize, out_f32;
  float over_scale;
};

template <int kLanes, int kV, bool kSoftmax, bool kF32>
__global__ __launch_bounds__(kRouteThreads) void moe_route_backward_kernel(const RouteBackwardArgs a) {
  constexpr int kMost = kLanes * kV, kSlots = kMaxTopK / kLanes;
  __shared__ float chosen[kRouteThreads / kLanes][kMost];  // d_j at the chosen experts, 0 elsewhere
  const int l = threadIdx.x % kLanes, group = threadIdx.x / kLanes, groups = blockDim.x / kLanes;
  const int E = a.E, k = a.k;
  float *const d_of = chosen[group];
  const float dloss = a.dloss != nullptr ? *a.dloss : 1.0f;
  float g[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int e = expert_of<kLanes>(l, v);
    g[v] = e < E ? a.slope[static_cast<int64_t>(blockIdx.y) * E + e] * dloss : 0.0f;
    d_of[e] = 0.0f;
  }
  wave_sync();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * groups;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * groups; first < a.S; first += stride) {
    const int64_t t = first + group, row = blockIdx.y * a.S + t;
    const bool here = t < a.S && a.ids[row * k] >= 0;
    float z[kV], s[kV], sum, top;
#pragma unroll
    for (int v = 0; v < kV; ++v) z[v] = -INFINITY;
    if (here) load_logits<kLanes, kV, kF32>(a.logits, row, E, l, z);
    scores<kLanes, kV, kSoftmax>(z, s, sum, top);
    if constexpr (!kSoftmax)
      if (__any(here && top < 0.0f)) raise_scores<kLanes, kV>(z, top, s, sum);
    const float r = 1.0f / sum;

    float w[kSlots], dw[kSlots], dot = 0.0f;
    int id[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int j = l + i * kLanes;
      id[i] = -1;
      if (i * kLanes >= k) break;
      id[i] = here && j < k ? a.ids[row * k + j] : -1;
      if (id[i] >= E) id[i] = -1;
      w[i] = dw[i] = 0.0f;
      if (id[i] >= 0) {
        w[i] = a.w[row * k + j];
        dw[i] = a.dw[row * k + j];
        dot = __builtin_fmaf(w[i], dw[i], dot);
      }
    }
    dot = across<kLanes>(dot, Add{});
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (id[i] >= 0) atomicAdd(&d_of[id[i]], w[i] * (a.normalize ? dw[i] - dot * a.over_scale : dw[i]));
    wave_sync();
    float along = 0.0f;  // sum of p g
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      s[v] = here ? s[v] : 0.0f;
      along = __builtin_fmaf(s[v], g[v], along);
    }
    along = across<kLanes>(along, Add{}) * r;
    if (kSoftmax && !a.normalize) along += dot;
    float dz[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const float d = __builtin_fmaf(s[v] * r, g[v] - along, d_of[expert_of<kLanes>(l, v)]);
      float rest = 1.0f;
      if (!kSoftmax) sigmoid(z[v], rest);
      dz[v] = here ? d * rest : 0.0f;
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (id[i] >= 0) d_of[id[i]] = 0.0f;
    wave_sync();
    if (t >= a.S) continue;
    const int64_t at = row * E;
#pragma unroll
    for (int j = 0; j < kV / 4; ++j) {
      const int e = 4 * (l + kLanes * j);
      if ((E & 3) == 0) {
        if (e >= E) break;
        if (a.out_f32)
          *reinterpret_cast<float4 *>(static_cast<float *>(a.dlogits) + at + e) =
              make_float4(dz[4 * j], dz[4 * j + 1], dz[4 * j + 2], dz[4 * j + 3]);
        else
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.dlogits) + at + e) =
              make_uint2(pack2_bf16(dz[4 * j], dz[4 * j + 1]), pack2_bf16(dz[4 * j + 2], dz[4 * j + 3]));
        continue;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (e + i >= E) break;
        if (a.out_f32)
          static_cast<float *>(a.dlogits)[at + e + i] = dz[4 * j + i];
        else
          static_cast<uint16_t *>(a.dlogits)[at + e + i] = static_cast<uint16_t>(pack2_bf16(dz[4 * j + i], 0.0f));
      }
    }
  }
}

// Lanes and values per lane for E experts: f(lanes, values) as integral constants.
template <class F>
void for_experts(int64_t E, F f) {
  using std::integral_constant;
  if (E <= 64)
    f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (E <= 128)
    f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (E <= 256)
    f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else
    f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

// Threads of a workgroup and workgroups per sequence of S tokens: one at the least, which writes the counts, the slope and the
// sums of a sequence without tokens too.
void route_grid(int64_t S, int64_t E, int &threads, int64_t &groups) {
  const int lanes = E <= 256 ? 16 : 64;
  const int64_t needed = (S * lanes + 63) / 64 * 64;
  threads = static_cast<int>(needed < kRouteThreads ? needed : kRouteThreads);
  if (threads == 0) threads = 64;
  const int64_t at_once = threads / lanes;
  groups = (S + at_once - 1) / at_once;
  if (groups > kRouteGroups) groups = kRouteGroups;
  if (groups == 0) groups = 1;
}

}  // namespace

int64_t moe_route_workspace(int64_t B, int64_t S, int64_t E) {
  int threads;
  int64_t groups;
  route_grid(S, E, threads, groups);
  return kHead + 8 * B * column_blocks(E) + 4 * B * groups * (2 * E + 2);
}

hipError_t launch_moe_route(const void *logits, bool f32, int64_t B, int64_t S, int64_t E, int64_t k, const float *bias,
                            const uint8_t *valid, bool softmax, bool normalize, float scale, double balance, int32_t *ids,
                            float *w, int32_t *counts, float *loss, float *slope, void *workspace, hipStream_t stream) {
  int threads;
  int64_t groups;
  route_grid(S, E, threads, groups);
  uint8_t *const ws = static_cast<uint8_t *>(workspace);
  const int64_t columns = column_blocks(E);
  RouteArgs a = {logits, bias,  valid, ids, w, counts, loss, slope, reinterpret_cast<uint32_t *>(ws),
                 reinterpret_cast<double *>(ws + kHead), reinterpret_cast<float *>(ws + kHead + 8 * B * columns),
                 B, S, static_cast<int>(E), static_cast<int>(k), normalize, scale, balance};
  const dim3 grid(static_cast<uint32_t>(groups), static_cast<uint32_t>(B)), block(threads);
  for_experts(E, [&](auto lanes, auto values) {
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    constexpr int kL = decltype(lanes)::value, kV = decltype(values)::value;
    if (softmax)
      f32 ? go(moe_route_kernel<kL, kV, true, true>) : go(moe_route_kernel<kL, kV, true, false>);
    else
      f32 ? go(moe_route_kernel<kL, kV, false, true>) : go(moe_route_kernel<kL, kV, false, false>);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (grid.x == 1 && grid.y == 1)) return e;
  hipLaunchKernelGGL(moe_route_sum_kernel, dim3(static_cast<uint32_t>(columns), static_cast<uint32_t>(B)), dim3(1024), 0,
                     stream, a, static_cast<int>(grid.x));
  return hipGetLastError();
}

hipError_t launch_moe_route_backward(const void *logits, bool f32, int64_t B, int64_t S, int64_t E, int64_t k,
                                     const int32_t *ids, const float *w, const float *dw, const float *slope,
                                     const float *dloss, bool softmax, bool normalize, float scale, void *dlogits,
                                     bool out_f32, hipStream_t stream) {
  int threads;
  int64_t groups;
  route_grid(S, E, threads, groups);
  const RouteBackwardArgs a = {logits, ids, w, dw, slope, dloss, dlogits, S, static_cast<int>(E), static_cast<int>(k),
                               normalize, out_f32, 1.0f / scale};
  const dim3 grid(static_cast<uint32_t>(groups), static_cast<uint32_t>(B)), block(threads);
  for_experts(E, [&](auto lanes, auto values) {
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    constexpr int kL = decltype(lanes)::value, kV = decltype(values)::value;
    if (softmax)
      f32 ? go(moe_route_backward_kernel<kL, kV, true, true>) : go(moe_route_backward_kernel<kL, kV, true, false>);
    else
      f32 ? go(moe_route_backward_kernel<kL, kV, false, true>) : go(moe_route_backward_kernel<kL, kV, false, false>);
  });
  return hipGetLastError();
}

}  // namespace fp8q
