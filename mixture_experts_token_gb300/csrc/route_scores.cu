// Routing by softmax or sigmoid scores with a balancing bias, groups of
// experts and renormalised weights, and its gradient; a warp a token.
//
//   c = s(logits) + bias; groups by the sum of their group_top largest c; the
//   k largest c of the groups kept; weights scale * s / (sum of the chosen s)
//
// Ranks must be those of 64-bit scores, or a near tie would send a token to
// another expert than the definition does.  So a row is ranked twice at most:
// in float32 with a bound on the error of every c, and, where two numbers
// whose order matters are nearer than that bound allows or a lane holds four of
// the chosen (1.5 and 2.6 rows in a thousand of random logits, 8 of 256 experts,
// by simulation), again in float64.
//
// Forward, in float32: lane i holds the i-th run of EPL consecutive experts,
// and its three largest c with the expert's place in the lowest bits.  k rounds
// of a warp maximum take the chosen in order, the lane that has one bringing its
// next.  Where a lane could have brought a fourth, or two that follow each other
// are nearer than the errors of c and of those bits allow, all that reach the
// k-th are put in a row and ranked in float64.  Without a bias, and where no sum
// of scores is compared, the logits rank, and the bits are the only error.
//
// Measured, 256 experts in 8 groups, 4 kept, 8 chosen, sigmoid with a bias:
// 65536 tokens 43.1 to 44.2 us (the bytes need 10.5; 505 instructions a token,
// issue slots 69% busy; of 490 at a step before, 80 were for the scores, 56 for
// the lanes' largest, 121 for the groups, 81 for the rounds, 82 to see that the
// order is sure, 68 for weights and stores; more CTAs an SM, or the bias read for
// each row, took 1 to 2 us longer), one token 3.6 us.  A row that float64 ranks
// adds 1.3 us where candidates are near, 2 to 3.6 where group sums are, 17 to 20
// in rank64().  Logits that are all equal send every row there: 65536 tokens then
// take 1.0 ms, without groups and a bias 0.30.  The gradient, 65536 tokens: 20.6
// us (73 MB must move, 10.8 us; 105 MB, 15.5 us, if HBM reads 64 bytes for a
// chosen logit).
#include <float.h>
#include <limits.h>
#include <math.h>

#include "launch.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxGroups = 64;
constexpr int kMaxGroupTop = 4;
constexpr float kLog2e = 1.4426950408889634f;

enum Rank { kByLogit, kBySigmoid, kBySoftmax };

struct Args {
  const float *logits, *bias;
  int32_t* idx;
  float* w;
  int32_t* status;
  int T, E, k, groups, top_groups, group_top;
  bool sigmoid, renorm, by_logit;
  float scale;
};

// The warp's largest and smallest (a NaN only if all are).
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_min(float v) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The weight of the chosen expert of logit l, in lanes where `chosen`, where
// a score or its share is below e^kFar: in float64, since float32 would lose
// it before the scale brings it back.  z and m as below.
constexpr float kFar = -80.0f;
__device__ __noinline__ float far_weight(const Args& a, bool chosen, float l,
                                         float m, float z) {
  // the score's logarithm
  double v = -INFINITY;
  if (chosen) {
    v = l;
    v = a.sigmoid ? fmin(v, 0.0) - log1p(exp(-fabs(v)))
                  : v - static_cast<double>(m) - log(static_cast<double>(z));
  }
  double top = 0.0, sum = 1.0;
  if (a.renorm) {
    top = v;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      top = fmax(top, __shfl_xor_sync(kAll, top, o));
    sum = warp_sum(chosen ? exp(v - top) : 0.0);
  }
  return chosen ? static_cast<float>(a.scale * (exp(v - top) / sum)) : 0.0f;
}

// The weight of the chosen expert of logit l, in lanes where `chosen`; z is
// the softmax's sum over all experts under the largest logit m.
template <int RANK>
__device__ __forceinline__ float weight(const Args& a, bool chosen, float l,
                                        float m, float z) {
  const bool sigmoid = RANK == kByLogit ? a.sigmoid : RANK == kBySigmoid;
  chosen = chosen && fabsf(l) <= FLT_MAX;
  float s = 0.0f;
  if (sigmoid) {
    if (__any_sync(kAll, chosen && l < kFar))
      return far_weight(a, chosen, l, m, z);
    const float x = expf(-fabsf(l));
    if (chosen) s = (l < 0.0f ? x : 1.0f) * rcp_fast(1.0f + x);
  } else {
    const float x = l - (a.renorm ? warp_max(chosen ? l : -FLT_MAX) : m);
    if (__any_sync(kAll, chosen && x < kFar))
      return far_weight(a, chosen, l, m, z);
    if (chosen) {
      s = expf(x);
      if (!a.renorm) s /= z;
    }
  }
  if (a.renorm) {
    // lanes past the k-th have nothing
    float sum = s;
    if (a.k > 8) {
      sum += __shfl_xor_sync(kAll, sum, 16);
      sum += __shfl_xor_sync(kAll, sum, 8);
    }
    sum += __shfl_xor_sync(kAll, sum, 4);
    sum += __shfl_xor_sync(kAll, sum, 2);
    sum += __shfl_xor_sync(kAll, sum, 1);
    s = sum > 0.0f ? __fdividef(s, sum) : 0.0f;
  }
  return a.scale * s;
}

// ------------------------------------------------------ in float64 -------
// The largest logit m and the softmax's sum z; finite logits alone.
__device__ void sums64(const Args& a, const float* row, int lane, float* m,
                       double* z) {
  float most = -INFINITY;
  for (int e = lane; e < a.E; e += 32)
    if (fabsf(row[e]) <= FLT_MAX) most = fmaxf(most, row[e]);
  *m = warp_max(most);
  double sum = 0.0;
  if (!a.sigmoid) {
    for (int e = lane; e < a.E; e += 32)
      if (fabsf(row[e]) <= FLT_MAX)
        sum += exp(static_cast<double>(row[e]) - static_cast<double>(*m));
    sum = warp_sum(sum);
  }
  *z = sum;
}
// c of expert e.  Experts that are not finite rank last.
__device__ double score64(const Args& a, const float* row, int e, float m,
                          double z) {
  const float l = row[e], b = a.bias ? a.bias[e] : 0.0f;
  if (!(fabsf(l) <= FLT_MAX) || !(fabsf(b) <= FLT_MAX)) return -INFINITY;
  if (a.by_logit) return l;
  const double x = l;
  const double s =
      a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - static_cast<double>(m)) / z;
  return s + b;
}
// What experts rank by: without a bias the logits, whose scores may round to
// the same number.
__device__ double rank_by64(const Args& a, const float* row, int e, float m,
                            double z) {
  if (a.bias) return score64(a, row, e, m, z);
  return fabsf(row[e]) <= FLT_MAX ? static_cast<double>(row[e]) : -INFINITY;
}
// Numbers as integers of the same order (no NaN; one zero).
__device__ __forceinline__ long long ordered64(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return b < 0 ? b ^ 0x7fffffffffffffffll : b;
}

// The rank of this lane's candidate e among those of the first `total` lanes.
__device__ __noinline__ int rank_candidates64(const Args& a, const float* row,
                                              int e, int total, int lane) {
  float m = 0.0f;
  double z = 1.0;
  if (a.bias && !a.sigmoid) sums64(a, row, lane, &m, &z);
  const long long v =
      lane < total ? ordered64(rank_by64(a, row, e, m, z)) : LLONG_MIN;
  int before = 0;
  for (int j = 0; j < total; ++j) {
    const long long other = __shfl_sync(kAll, v, j);
    const int oe = __shfl_sync(kAll, e, j);
    before += other > v || (other == v && oe < e);
  }
  return before;
}

// The largest of the lanes' numbers.
__device__ __forceinline__ long long warp_max64(long long v) {
  const int hi = __reduce_max_sync(kAll, static_cast<int>(v >> 32));
  const uint32_t lo = __reduce_max_sync(
      kAll, static_cast<int>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<long long>(hi) << 32 | lo;
}

// Whether the group of lane / lanes takes part, from the float64 sums of those
// experts that the groups' largest c can be: one of the first `total` lanes
// each, e its expert.  (Equal sums: the lower group.)
__device__ __noinline__ bool keep_groups64(const Args& a, const float* row,
                                           int e, int total, int lane,
                                           int lanes) {
  float m = 0.0f;
  double z = 1.0;
  if (!a.sigmoid) sums64(a, row, lane, &m, &z);
  const int size = a.E / a.groups;
  long long v = LLONG_MIN;
  if (lane < total) v = ordered64(score64(a, row, e, m, z));
  const int mine = lane < total ? e / size : -1;
  long long sum = LLONG_MIN;  // of group `lane`
  for (int g = 0; g < a.groups; ++g) {
    long long left = mine == g ? v : LLONG_MIN;
    double t = 0.0;
    for (int j = 0; j < a.group_top; ++j) {
      const long long best = warp_max64(left);
      if (lane == __ffs(__ballot_sync(kAll, left == best)) - 1)
        left = LLONG_MIN;
      t += __longlong_as_double(best < 0 ? best ^ 0x7fffffffffffffffll : best);
    }
    if (lane == g) sum = ordered64(t);
  }
  int before = 0;
  for (int g = 0; g < a.groups; ++g) {
    const long long other = __shfl_sync(kAll, sum, g);
    before += other > sum || (other == sum && g < lane);
  }
  const uint32_t keep =
      __ballot_sync(kAll, lane < a.groups && before < a.top_groups);
  return lane / lanes < a.groups && keep >> (lane / lanes) & 1;
}

// Ranks a row anew, groups and experts; lane j returns the j-th expert.  c:
// room for the row's E numbers, as integers of their order.  Late rows of a
// call wait for nothing else, so what counts is the time of one: float64
// instructions are few and side by side.
__device__ __noinline__ int rank64(const Args& a, const float* row, int lane,
                                   long long* c, float* max_logit,
                                   float* sum) {
  bool bad = false;
  for (int e = lane; e < a.E; e += 32)
    bad |= !(fabsf(row[e]) <= FLT_MAX) ||
           (a.bias && !(fabsf(a.bias[e]) <= FLT_MAX));
  if (__any_sync(kAll, bad) && lane == 0 && a.status)
    atomicOr(a.status, MOE_DEV_NONFINITE);
  float m;
  double z;
  sums64(a, row, lane, &m, &z);
  *max_logit = m;
  *sum = static_cast<float>(z);

  // the groups that take part, a lane for two of them
  unsigned long long keep = ~0ull;
  const int size = a.E / a.groups;
  __syncwarp();
  if (a.top_groups < a.groups) {
#pragma unroll 4
    for (int e = lane; e < a.E; e += 32)
      c[e] = ordered64(score64(a, row, e, m, z));
    __syncwarp();
    double total[2] = {-INFINITY, -INFINITY};
    for (int g = 0; g < a.groups; ++g) {
      // its group_top largest, one after another; equal ones one by one
      double t = 0.0;
      long long under = LLONG_MAX;  // none above it is left
      int taken = 0;                // of those equal to it
      for (int j = 0; j < a.group_top; ++j) {
        long long best = LLONG_MIN;
        int equal = 0;
        for (int e = g * size + lane; e < (g + 1) * size; e += 32) {
          const long long v = c[e];
          if (v < under) best = max(best, v);
          equal += v == under;
        }
        if (__reduce_add_sync(kAll, equal) > taken) {
          ++taken;
        } else {
          under = warp_max64(best);
          taken = 1;
        }
        const long long bits =
            under < 0 ? under ^ 0x7fffffffffffffffll : under;
        t += __longlong_as_double(bits);
      }
      if (lane == (g & 31)) total[g >> 5] = t;
    }
    const long long mine[2] = {ordered64(total[0]), ordered64(total[1])};
    int before[2] = {0, 0};
    for (int g = 0; g < a.groups; ++g) {
      const long long t =
          __shfl_sync(kAll, g < 32 ? mine[0] : mine[1], g & 31);
      for (int h = 0; h < 2; ++h)
        before[h] += t > mine[h] || (t == mine[h] && g < h * 32 + lane);
    }
    keep = __ballot_sync(kAll, lane < a.groups && before[0] < a.top_groups);
    keep |= static_cast<unsigned long long>(__ballot_sync(
                kAll, 32 + lane < a.groups && before[1] < a.top_groups))
            << 32;
  }

  const int per = (a.E + 31) / 32, first = lane * per;
  uint32_t left = 0;  // this lane's experts that may be chosen yet
  __syncwarp();  // c is written anew
  for (int i = 0; i < per; ++i) {
    const int e = first + i;
    if (e < a.E && keep >> (e / size) & 1) {
      if (!a.bias || a.top_groups == a.groups)  // else c holds it already
        c[e] = ordered64(rank_by64(a, row, e, m, z));
      left |= 1u << i;
    }
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    long long best = LLONG_MIN;
    int at = kMaxExperts;
    for (int i = 0; i < per; ++i)
      if (left >> i & 1) {
        const long long v = c[first + i];
        if (at == kMaxExperts || v > best) {
          best = v;
          at = first + i;
        }
      }
    const long long top = warp_max64(best);
    const int e = __reduce_min_sync(
        kAll, best == top ? static_cast<unsigned>(at) : kMaxExperts + 0u);
    if (e >= first && e < first + per) left &= ~(1u << (e - first));
    if (lane == j) mine = e;
  }
  __syncwarp();
  return mine;
}

// ------------------------------------------------------ in float32 -------
// Experts e0 .. e0 + EPL - 1 of a row; -infinity past the last.
template <int EPL, bool FULL>
__device__ __forceinline__ void load_row(const float* row, int e0, int E,
                                         bool wide, float (&c)[EPL]) {
  if constexpr (EPL % 4 == 0) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4) {
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (FULL || e0 + i < E)
          v = *reinterpret_cast<const float4*>(row + e0 + i);
        c[i] = v.x, c[i + 1] = v.y, c[i + 2] = v.z, c[i + 3] = v.w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    c[i] = FULL || e0 + i < E ? row[e0 + i] : -INFINITY;
}

// c of a logit l; m and inv: the softmax's largest logit and 1 / its sum.
template <int RANK>
__device__ __forceinline__ float rank_by(float l, float bias, float m,
                                         float inv) {
  if (RANK == kByLogit) return l;
  const float s = RANK == kBySigmoid
                      ? rcp_fast(1.0f + exp2_fast(-kLog2e * l))
                      : exp2_fast((l - m) * kLog2e) * inv;
  return s + bias;
}

// A lane's three largest of v, with the place in the lowest bits.
template <int EPL>
struct Top {
  float a = -INFINITY, b = -INFINITY, c = -INFINITY;
  static __device__ __forceinline__ float key(float v, int i) {
    return __uint_as_float(
        (__float_as_uint(fmaxf(v, -FLT_MAX)) & ~(EPL - 1u)) | i);
  }
  __device__ __forceinline__ Top() {}
  __device__ __forceinline__ explicit Top(const float (&v)[EPL]) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      float k = key(v[i], i);
      const float under = fminf(a, k);
      a = fmaxf(a, k);
      if (EPL < 2) continue;
      k = under;
      const float third = fminf(b, k);
      b = fmaxf(b, k);
      if (EPL > 2) c = fmaxf(c, third);
    }
  }
};
// What a key may be off by, of its magnitude: EPL - 1 units in the last place.
template <int EPL>
constexpr float kKeyErr = EPL * 1.1920929e-7f;

// Puts the experts of the lanes' hits into the list, up to 32, in any order;
// how many there are (33 or more: too many).
__device__ __forceinline__ int collect(uint32_t hits, int e0, int lane,
                                       int* list) {
  int total = 0;
  __syncwarp();
#pragma unroll 1
  for (uint32_t any; (any = __ballot_sync(kAll, hits != 0)) != 0;) {
    const int at = total + __popc(any & ((1u << lane) - 1));
    total += __popc(any);
    if (hits != 0 && at < 32) list[at] = e0 + __ffs(hits) - 1;
    if (total > 32) break;
    hits &= hits - 1;
  }
  __syncwarp();
  return total;
}

// FULL: E is 32 EPL.
template <int EPL, int RANK, bool FULL>
__global__ void __launch_bounds__(kThreads, EPL <= 8 ? 8 : 4)
    scores_kernel(const Args a) {
  // the chosen, a key and its lane's first expert; candidates of a closer look;
  // the row's numbers, where groups are not whole lanes and in rank64()
  __shared__ float2 chosen[kWarps][32];
  __shared__ int cand_e[kWarps][32];
  extern __shared__ long long row_c[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long* mine64 = row_c + warp * (32 * EPL);
  const int size = a.E / a.groups;
  const bool select = a.top_groups < a.groups;
  // groups of whole lanes, a power of two of them
  const int lanes = size / EPL;
  const bool whole = size % EPL == 0 && (lanes & (lanes - 1)) == 0 &&
                     a.group_top <= 2;
  const int e0 = lane * EPL;
  const bool wide = EPL % 4 == 0 && (FULL || a.E % 4 == 0) &&
                    (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
  launch::wait_for_previous();
  launch::let_next_start();
  float bias[EPL], most_bias = 0.0f;
  if (RANK != kByLogit) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      bias[i] = a.bias && e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
      // one that is not finite sends every row to rank64()
      most_bias = fabsf(bias[i]) <= FLT_MAX ? fmaxf(most_bias, fabsf(bias[i]))
                                            : INFINITY;
    }
    most_bias = warp_max(most_bias);
  }
  const long long step = gridDim.x * static_cast<long long>(kWarps);
#pragma unroll 1
  for (long long t = blockIdx.x * static_cast<long long>(kWarps) + warp;
       t < a.T; t += step) {
    const float* row = a.logits + t * a.E;
    float c[EPL];
    load_row<EPL, FULL>(row, e0, a.E, wide, c);
    float nan = RANK != kByLogit && most_bias == INFINITY ? NAN : 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (FULL || e0 + i < a.E) nan = fmaf(c[i], 0.0f, nan);
    bool again = nan != 0.0f;  // a logit or a bias is not finite

    // scores, and the most that a c may be off by
    float m = 0.0f, z = 1.0f, inv = 1.0f, err = 0.0f, most = 0.0f;
    if (RANK == kBySoftmax || (RANK == kByLogit && !a.sigmoid && !a.renorm)) {
      m = c[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) m = fmaxf(m, c[i]);
      m = warp_max(m);
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float x = exp2_fast((c[i] - m) * kLog2e);
        if (RANK == kBySoftmax) c[i] = x;
        part += x;
      }
      z = warp_sum(part);
      inv = rcp_fast(z);
    }
    if (RANK != kByLogit) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        c[i] = RANK == kBySoftmax ? c[i] * inv + bias[i]
                                  : rank_by<RANK>(c[i], bias[i], m, inv);
        if (!FULL && e0 + i >= a.E) c[i] = -INFINITY;
      }
      // The sigmoid: 2^-22 of the exponential and what its argument's rounding
      // gives (a third of 2^-24), weighed by s (1 - s) <= 1/4, an ulp of the
      // reciprocal and half of one of the sum before it: below 2^-21.  The
      // softmax, of the largest score: its sum of up to 1024 terms is off by
      // 2^-22, by 17 2^-24 from the arguments (far terms: 10 bits of them at
      // most weigh) and by 37 2^-24 from adding: below 2^-18.  Adding the
      // bias: half an ulp.
      most = RANK == kBySoftmax ? inv : 1.0f;
      err = (RANK == kBySoftmax ? 3.8146973e-6f : 4.7683716e-7f) * most +
            1.1920929e-7f * (most + most_bias);
    }

    Top<EPL> top(c);
    bool kept = true;
    if (select) {
      // sums of n c are off by n errors, and adding them by n (n - 1) / 2
      const float group_err = a.group_top * (a.group_top + 1) * err;
      if (whole) {
        float g1 = top.a, g2 = top.b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          if (o >= lanes) break;
          const float o1 = __shfl_xor_sync(kAll, g1, o);
          const float o2 = __shfl_xor_sync(kAll, g2, o);
          g2 = fmaxf(fminf(g1, o1), fmaxf(g2, o2));
          g1 = fmaxf(g1, o1);
        }
        // (lanes past the last expert are behind all groups)
        float o = FULL || e0 < a.E ? (a.group_top == 2 ? g1 + g2 : g1)
                                   : -INFINITY;
        kept = false;
        float last = 0.0f;
#pragma unroll 4
        for (int g = 0; g < a.top_groups; ++g) {
          last = warp_max(o);
          if (o == last) {
            kept = true;
            o = -INFINITY;
          }
        }
        const float out = warp_max(o);
        // equal sums, or sums that the errors may have exchanged
        const float keys =
            kKeyErr<EPL> * (RANK == kByLogit
                                ? fabsf(last) + fabsf(out)
                                : 2 * a.group_top * (most + most_bias));
        if (__popc(__ballot_sync(kAll, kept)) != a.top_groups * lanes ||
            !(last - out > group_err + keys + FLT_MIN)) {
          const float g = a.group_top == 2 ? g2 : g1;
          const float least =
              g - 2.0f * (err + kKeyErr<EPL> * fabsf(g) + FLT_MIN);
          // (behind the last expert c and `least` are both -infinity)
          uint32_t hits = 0;
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            if ((FULL || e0 + i < a.E) && c[i] >= least) hits |= 1u << i;
          const int n = collect(hits, e0, lane, cand_e[warp]);
          if (n > 32)
            again = true;
          else
            kept = keep_groups64(a, row, lane < n ? cand_e[warp][lane] : 0, n,
                                 lane, lanes);
        }
        if (!kept) top = Top<EPL>();
      } else {
        // a lane a group (or two), over the row's c in shared memory
        float* rc = reinterpret_cast<float*>(mine64);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; ++i) rc[e0 + i] = c[i];
        __syncwarp();
        float total[2];
        for (int h = 0; h < 2; ++h) {
          const int g = h * 32 + lane;
          total[h] = -INFINITY;
          if (g >= a.groups) continue;
          float top[kMaxGroupTop];
#pragma unroll
          for (int j = 0; j < kMaxGroupTop; ++j) top[j] = -INFINITY;
          for (int e = g * size; e < (g + 1) * size; ++e) {
            float v = rc[e];
#pragma unroll
            for (int j = 0; j < kMaxGroupTop; ++j) {
              const float hi = fmaxf(top[j], v);
              v = fminf(top[j], v);
              top[j] = hi;
            }
          }
          total[h] = top[0];
#pragma unroll
          for (int j = 1; j < kMaxGroupTop; ++j)
            if (j < a.group_top) total[h] += top[j];
        }
        int before[2] = {0, 0};
        for (int g = 0; g < a.groups; ++g) {
          const float other =
              __shfl_sync(kAll, g < 32 ? total[0] : total[1], g & 31);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            before[h] += other > total[h] ||
                         (other == total[h] && g < h * 32 + lane);
        }
        const bool k0 = lane < a.groups && before[0] < a.top_groups;
        const bool k1 = 32 + lane < a.groups && before[1] < a.top_groups;
        if (RANK != kByLogit) {
          const float last = warp_min(
              fminf(k0 ? total[0] : INFINITY, k1 ? total[1] : INFINITY));
          const float out = warp_max(
              fmaxf(lane < a.groups && !k0 ? total[0] : -INFINITY,
                    32 + lane < a.groups && !k1 ? total[1] : -INFINITY));
          again |= !(last - out > group_err);
        }
        const uint32_t low = __ballot_sync(kAll, k0);
        const uint32_t high = __ballot_sync(kAll, k1);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int g = (e0 + i) / size;
          if (g >= a.groups || !((g < 32 ? low >> g : high >> (g - 32)) & 1))
            c[i] = -INFINITY;
        }
        top = Top<EPL>(c);
      }
    }

    // The largest left in the warp, k times: its lane brings the next.
    float reached = 0.0f, behind = -INFINITY;
    {
      float o1 = top.a, o2 = top.b, o3 = top.c;
      __syncwarp();
#pragma unroll 4
      for (int j = 0; j < a.k; ++j) {
        reached = warp_max(o1);
        if (o1 == reached) {
          chosen[warp][j] = make_float2(o1, __int_as_float(e0));
          o1 = o2;
          o2 = o3;
          o3 = -INFINITY;
        }
      }
      behind = fmaxf(warp_max(o1), -FLT_MAX);
    }
    again |= !(reached > -3.4e38f);  // fewer than k

    int e = 0;
    float l = 0.0f;
    if (!__any_sync(kAll, again)) {
      // what is left out below this is surely behind the k-th
      const float bar = fmaxf(
          reached - 2.0f * (err + kKeyErr<EPL> * fabsf(reached) + FLT_MIN),
          -FLT_MAX);
      // Keys that reach the k-th, equal ones among them: as many as were chosen.
      // A lane that brought three may have others, which must not come near.
      int n = (top.a >= reached) + (top.b >= reached) + (top.c >= reached);
      if (EPL > 3 && __any_sync(kAll, n == 3)) {
        if (n == 3) {
          n = 0;
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            n += kept && Top<EPL>::key(c[i], i) >= bar;
        }
      }
      __syncwarp();
      const float2 own = chosen[warp][lane];
      float next = __shfl_down_sync(kAll, own.x, 1);
      if (lane == a.k - 1) next = behind;
      e = min(__float_as_int(own.y) +
                  static_cast<int>(__float_as_uint(own.x) & (EPL - 1u)),
              a.E - 1);  // (of lanes that have one no change)
      // nearer than the errors allow, before or among the k chosen
      const bool near =
          lane < a.k &&
          !(own.x - next > 2.0f * err + FLT_MIN +
                               kKeyErr<EPL> * (fabsf(own.x) + fabsf(next)));
      if (__any_sync(kAll, near) || __reduce_add_sync(kAll, n) != a.k) {
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (c[i] >= bar) hits |= 1u << i;
        if (!kept) hits = 0;
        const int total = collect(hits, e0, lane, cand_e[warp]);
        again = total > 32 || total < a.k;
        if (!again) {
          const int mine = lane < total ? cand_e[warp][lane] : 0;
          const int rank = rank_candidates64(a, row, mine, total, lane);
          __syncwarp();
          if (lane < total) cand_e[warp][rank] = mine;
          __syncwarp();
          e = cand_e[warp][lane];
        }
      }
    }
    if (!__any_sync(kAll, again)) {
      l = lane < a.k ? row[e] : 0.0f;
    } else {
      e = rank64(a, row, lane, mine64, &m, &z);
      l = lane < a.k ? row[e] : 0.0f;
      if (lane < a.k && a.bias && !(fabsf(a.bias[e]) <= FLT_MAX)) l = INFINITY;
    }
    const float w = weight<RANK>(a, lane < a.k, l, m, z);
    if (lane < a.k) {
      a.idx[t * a.k + lane] = e;
      a.w[t * a.k + lane] = w;
    }
  }
}

// ---------------------------------------------------------- backward -----
struct BackArgs {
  const float* logits;
  const int32_t* idx;
  const float* dw;
  float* dlogits;
  int T, E, k;
  bool renorm;
  float scale;
};

// A chosen expert's gradient where a weight, one less a score or the weight's
// gradient is out of float32's range on the way: in float64, and with the
// sigmoid's 1 - s in it.  All lanes of the warp.
template <bool SIGMOID, int LANES>
__device__ __noinline__ float far_gradient(const BackArgs& a, bool finite,
                                           float l, float d, float m,
                                           float z) {
  const auto token_sum = [](double v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
  };
  double v = -INFINITY;  // the score's logarithm
  if (finite) {
    v = l;
    v = SIGMOID ? fmin(v, 0.0) - log1p(exp(-fabs(v)))
                : v - static_cast<double>(m) - log(static_cast<double>(z));
  }
  double top = 0.0;
  if (a.renorm) {
    top = v;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
      top = fmax(top, __shfl_xor_sync(kAll, top, o));
  }
  double w = finite ? exp(v - top) : 0.0;
  double g = finite ? static_cast<double>(a.scale) * d : 0.0;
  if (a.renorm) {
    const double sum = token_sum(w);
    if (finite) w /= sum;
    g -= token_sum(w * g);
  }
  g *= w;
  if (SIGMOID && finite) g /= 1.0 + exp(static_cast<double>(l));
  return static_cast<float>(g);
}
// f e^x, x <= 0, also where e^x alone is below float32's range.
__device__ __forceinline__ float times_exp(float f, float x) {
  const float root = expf(0.5f * x);
  return f * root * root;
}

// A chosen expert a lane, LANES lanes a token and so 32 / LANES tokens a warp.
// With sigmoid scores the row is zero but for the chosen; with softmax scores
// every lane also has its share of the row, one token after another.
template <bool SIGMOID, int LANES>
__global__ void __launch_bounds__(kThreads) scores_backward_kernel(
    const BackArgs a) {
  constexpr int kTokens = 32 / LANES;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = lane / LANES, j = lane % LANES;
  const bool wide =
      a.E % 4 == 0 &&
      ((reinterpret_cast<uintptr_t>(a.logits) |
        reinterpret_cast<uintptr_t>(a.dlogits)) & 15) == 0;
  const auto token_sum = [](float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
  };
  launch::wait_for_previous();
  launch::let_next_start();
  const long long step =
      gridDim.x * static_cast<long long>(kWarps) * kTokens;
  long long t0 = (blockIdx.x * static_cast<long long>(kWarps) + warp) *
                 kTokens;
  // An expert of no lane's choice, and no other lane's, where there is none.
  const auto choice = [&](long long first, int* e, float* d) {
    *e = -1 - lane;
    *d = 0.0f;
    const long long t = first + tok;
    if (t < a.T && j < a.k) {
      const int i = a.idx[t * a.k + j];
      *d = a.dw[t * a.k + j];
      if (i >= 0 && i < a.E) *e = i;
    }
  };
  const auto logit = [&](long long first, int e) {
    return e >= 0 ? a.logits[(first + tok) * a.E + e] : 0.0f;
  };
  // the next tokens' choices and their logits come while these are worked on
  int next_e;
  float next_d, next_l;
  choice(t0, &next_e, &next_d);
  next_l = logit(t0, next_e);
  for (; t0 < a.T; t0 += step) {
    const long long t = t0 + tok;
    const int here = static_cast<int>(min(static_cast<long long>(kTokens),
                                          a.T - t0));
    const int e = next_e;
    const float l = next_l, d = next_d;
    choice(t0 + step, &next_e, &next_d);
    float m = 0.0f, z = 1.0f;
    if (SIGMOID) {
      // zeros now, while the chosen logits come
      float* out = a.dlogits + t0 * a.E;
      const long long n = static_cast<long long>(here) * a.E;
      if (wide)
        for (long long i = lane * 4; i < n; i += 128)
          *reinterpret_cast<float4*>(out + i) =
              make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      else
        for (long long i = lane; i < n; i += 32) out[i] = 0.0f;
    } else {
      for (int r = 0; r < here; ++r) {
        const float* row = a.logits + (t0 + r) * a.E;
        float most = -FLT_MAX;
        for (int i = lane; i < a.E; i += 32) {
          const float v = row[i];
          if (fabsf(v) <= FLT_MAX) most = fmaxf(most, v);
        }
        most = warp_max(most);
        float sum = 0.0f;
        for (int i = lane; i < a.E; i += 32) {
          const float v = row[i];
          if (fabsf(v) <= FLT_MAX) sum += expf(v - most);
        }
        sum = warp_sum(sum);
        if (tok == r) {
          m = most;
          z = sum;
        }
      }
    }
    next_l = logit(t0 + step, next_e);
    const bool finite = e >= 0 && fabsf(l) <= FLT_MAX;
    // the weight over scale, as the forward has it
    float top = finite ? l : -FLT_MAX;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
      top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    float w = 0.0f;
    if (finite) {
      if (SIGMOID)
        w = expf(fminf(l, 0.0f) - (a.renorm ? fminf(top, 0.0f) : 0.0f)) /
            (1.0f + expf(-fabsf(l)));
      else
        w = a.renorm ? expf(l - top) : expf(l - m) / z;
    }
    if (a.renorm) {
      const float sum = token_sum(w);
      w = sum > 0.0f ? w / sum : 0.0f;
    }
    float g = finite ? a.scale * d : 0.0f;
    const uint32_t mine = (LANES == 32 ? kAll : (1u << LANES) - 1)
                          << (tok * LANES);
    const uint32_t far_lanes = __ballot_sync(
        kAll, finite && (w < 1e-30f || fabsf(g) > 1e30f ||
                         (SIGMOID && fabsf(l) > -kFar)));
    // (by the token: what others in the warp have changes no bit of it)
    const bool far = far_lanes & mine;
    g *= w;
    if (a.renorm) g -= w * token_sum(g);
    if (far_lanes != 0) {
      const float f = far_gradient<SIGMOID, LANES>(a, finite, l, d, m, z);
      if (far) g = f;
    }
    const float all = SIGMOID ? 0.0f : token_sum(g);
    // an index that stands twice has the sum of both
    const uint32_t same =
        __match_any_sync(kAll, e) & mine & ~(1u << lane);
    if (__any_sync(kAll, e >= 0 && same != 0)) {
      float sum = 0.0f;
      for (int i = 0; i < LANES; ++i) {
        const float other = __shfl_sync(kAll, g, tok * LANES + i);
        if (tok * LANES + i == lane || same >> (tok * LANES + i) & 1)
          sum += other;
      }
      g = sum;
    }
    if (!SIGMOID) {
      for (int r = 0; r < here; ++r) {
        const float* row = a.logits + (t0 + r) * a.E;
        float* out = a.dlogits + (t0 + r) * a.E;
        const float most = __shfl_sync(kAll, m, r * LANES);
        const float f = __shfl_sync(kAll, -all / z, r * LANES);
        if (wide) {
          for (int i = lane * 4; i < a.E; i += 128) {
            const float4 v = *reinterpret_cast<const float4*>(row + i);
            float4 o;
            o.x = fabsf(v.x) <= FLT_MAX ? times_exp(f, v.x - most) : 0.0f;
            o.y = fabsf(v.y) <= FLT_MAX ? times_exp(f, v.y - most) : 0.0f;
            o.z = fabsf(v.z) <= FLT_MAX ? times_exp(f, v.z - most) : 0.0f;
            o.w = fabsf(v.w) <= FLT_MAX ? times_exp(f, v.w - most) : 0.0f;
            *reinterpret_cast<float4*>(out + i) = o;
          }
        } else {
          for (int i = lane; i < a.E; i += 32) {
            const float v = row[i];
            out[i] = fabsf(v) <= FLT_MAX ? times_exp(f, v - most) : 0.0f;
          }
        }
      }
    }
    __syncwarp();  // the chosen are written over what other lanes wrote
    if (finite)
      a.dlogits[t * a.E + e] = !SIGMOID ? g - times_exp(all / z, l - m)
                               : far    ? g
                                        : g * (1.0f / (1.0f + expf(l)));
  }
}

template <bool SIGMOID, int LANES>
cudaError_t launch_backward_of(const BackArgs& a, cudaStream_t s) {
  constexpr auto kernel = scores_backward_kernel<SIGMOID, LANES>;
  constexpr int kTokens = kWarps * 32 / LANES;  // of a CTA
  launch::Device d;
  int per_sm = 1;
  cudaError_t e = launch::device(&d);
  if (e == cudaSuccess)
    e = launch::ctas_per_sm<kernel>(d, kThreads, 0, &per_sm);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(std::min<long long>(
      (static_cast<long long>(a.T) + kTokens - 1) / kTokens,
      static_cast<long long>(per_sm) * d.sms));
  return launch::overlapping(kernel, grid, kThreads, 0, s, a);
}
template <bool SIGMOID>
cudaError_t launch_backward(const BackArgs& a, cudaStream_t s) {
  return a.k <= 4    ? launch_backward_of<SIGMOID, 4>(a, s)
         : a.k <= 8  ? launch_backward_of<SIGMOID, 8>(a, s)
         : a.k <= 16 ? launch_backward_of<SIGMOID, 16>(a, s)
                     : launch_backward_of<SIGMOID, 32>(a, s);
}

bool options_ok(const moe_config_t& c, const moe_route_scores_t* o) {
  if (o == nullptr) return false;
  if (o->score != MOE_SCORE_SOFTMAX && o->score != MOE_SCORE_SIGMOID)
    return false;
  if (o->renorm != 0 && o->renorm != 1) return false;
  if (!(fabsf(o->scale) <= FLT_MAX)) return false;
  if (o->groups < 1 || o->groups > kMaxGroups || c.E % o->groups != 0 ||
      o->top_groups < 1 || o->top_groups > o->groups)
    return false;
  const int size = c.E / o->groups;
  return o->group_top >= 1 && o->group_top <= std::min(kMaxGroupTop, size) &&
         static_cast<long long>(o->top_groups) * size >= c.k;
}

template <int EPL, int RANK, bool FULL>
cudaError_t launch_scores(const Args& a, cudaStream_t s) {
  constexpr auto kernel = scores_kernel<EPL, RANK, FULL>;
  constexpr int kBytes = kWarps * 32 * EPL * sizeof(long long);
  static_assert(kBytes + kWarps * 384 <= 48 * 1024, "no larger than any CTA's");
  launch::Device d;
  int per_sm = 1;
  cudaError_t e = launch::device(&d);
  if (e == cudaSuccess)
    e = launch::ctas_per_sm<kernel>(d, kThreads, kBytes, &per_sm);
  if (e != cudaSuccess) return e;
  // CTAs that stay, so that a warp reads the bias once
  const unsigned grid = static_cast<unsigned>(std::min<long long>(
      (static_cast<long long>(a.T) + kWarps - 1) / kWarps,
      static_cast<long long>(per_sm) * d.sms));
  return launch::overlapping(kernel, grid, kThreads, kBytes, s, a);
}
template <int EPL, bool FULL>
cudaError_t launch_rank(const Args& a, cudaStream_t s) {
  return a.by_logit  ? launch_scores<EPL, kByLogit, FULL>(a, s)
         : a.sigmoid ? launch_scores<EPL, kBySigmoid, FULL>(a, s)
                     : launch_scores<EPL, kBySoftmax, FULL>(a, s);
}
template <int EPL>
cudaError_t launch_epl(const Args& a, cudaStream_t s) {
  return a.E == 32 * EPL ? launch_rank<EPL, true>(a, s)
                         : launch_rank<EPL, false>(a, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_route_scores(const moe_config_t* cfg,
                              const moe_route_scores_t* opt,
                              const float* logits, const float* bias,
                              int32_t* topk_idx, float* topk_w,
                              int32_t* status_word, moe_stream_t stream) {
  const moe_status_t st = validate(cfg);
  if (st != MOE_OK) return st;
  if (!options_ok(*cfg, opt) || (bias != nullptr && !ok_ptr(bias, false)))
    return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!ok_ptr(logits, false) || !ok_ptr(topk_idx, false) ||
      !ok_ptr(topk_w, false))
    return MOE_ERR_INVALID_ARG;
  Args a = {};
  a.logits = logits;
  a.bias = bias;
  a.idx = topk_idx;
  a.w = topk_w;
  a.status = status_word;
  a.T = cfg->T;
  a.E = cfg->E;
  a.k = cfg->k;
  a.groups = opt->groups;
  a.top_groups = opt->top_groups;
  a.group_top = opt->group_top;
  a.sigmoid = opt->score == MOE_SCORE_SIGMOID;
  a.renorm = opt->renorm != 0;
  a.scale = opt->scale;
  // the scores rise with the logits; only sums and biases need their values
  a.by_logit = bias == nullptr &&
               (opt->top_groups == opt->groups || opt->group_top == 1);
  const int per = (cfg->E + 31) / 32;
  cudaError_t e;
  if (per <= 1)
    e = launch_epl<1>(a, stream);
  else if (per <= 2)
    e = launch_epl<2>(a, stream);
  else if (per <= 4)
    e = launch_epl<4>(a, stream);
  else if (per <= 8)
    e = launch_epl<8>(a, stream);
  else if (per <= 16)
    e = launch_epl<16>(a, stream);
  else
    e = launch_epl<32>(a, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_route_scores_backward(const moe_config_t* cfg,
                                       const moe_route_scores_t* opt,
                                       const float* logits,
                                       const int32_t* topk_idx,
                                       const float* dtopk_w, float* dlogits,
                                       moe_stream_t stream) {
  const moe_status_t st = validate(cfg);
  if (st != MOE_OK) return st;
  if (!options_ok(*cfg, opt)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!ok_ptr(logits, false) || !ok_ptr(topk_idx, false) ||
      !ok_ptr(dtopk_w, false) || !ok_ptr(dlogits, false) ||
      dlogits == logits)  // a row is written while it is read
    return MOE_ERR_INVALID_ARG;
  const BackArgs a = {logits, topk_idx, dtopk_w, dlogits, cfg->T, cfg->E,
                      cfg->k, opt->renorm != 0, opt->scale};
  const cudaError_t e = opt->score == MOE_SCORE_SIGMOID
                            ? launch_backward<true>(a, stream)
                            : launch_backward<false>(a, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
