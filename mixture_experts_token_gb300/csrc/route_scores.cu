// Routing by softmax or sigmoid scores with a balancing bias, groups of
// experts and renormalised weights, and its gradient; a warp a token.
//
//   c = s(logits) + bias; groups by the sum of their group_top largest c; the
//   k largest c of the groups kept; weights scale * s / (sum of the chosen s)
//
// Ranks must be those of 64-bit scores, or a near tie would send a token to
// another expert than the definition does.  So a row is ranked twice at most:
// in float32 with a bound on the error of every c, and, where two numbers
// whose order matters are nearer than that bound allows (about one row in a
// thousand), again in float64.
//
// Forward, in float32: lane i holds the i-th run of EPL consecutive experts,
// so that equal values go to the lower lane.  Each lane's two largest c give,
// in k rounds of a warp maximum, a threshold that at least k values reach; the
// few that do (and those within the error of it) are put in a row in shared
// memory in the order of their experts, one to a lane, and each counts those
// before it.  That is its rank: no list is sorted and no lane's values are
// searched again.  Without a bias, and where no sum of scores is compared, the
// logits rank, and there is no error to allow for.
#include <float.h>
#include <math.h>

#include "internal.h"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 256;
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

__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ float warp_max(float v) {
  return unordered(__reduce_max_sync(kAll, ordered(v)));
}
__device__ __forceinline__ float warp_min(float v) {
  return unordered(__reduce_min_sync(kAll, ordered(v)));
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

// The weight of the chosen expert of logit l, in lanes where `chosen`; z is
// the softmax's sum over all experts under the largest logit m.  Sums of
// chosen scores are taken relative to the largest of them, so that they do not
// vanish where all are small.
__device__ __forceinline__ float weight(const Args& a, bool chosen, float l,
                                        float m, float z) {
  chosen = chosen && fabsf(l) <= FLT_MAX;
  const float top = a.renorm ? warp_max(chosen ? l : -FLT_MAX) : 0.0f;
  float s = 0.0f;
  if (chosen) {
    if (a.sigmoid)
      s = expf(fminf(l, 0.0f) - (a.renorm ? fminf(top, 0.0f) : 0.0f)) /
          (1.0f + expf(-fabsf(l)));
    else
      s = a.renorm ? expf(l - top) : expf(l - m) / z;
  }
  if (a.renorm) {
    const float sum = warp_sum(s);
    s = sum > 0.0f ? s / sum : 0.0f;
  }
  return a.scale * s;
}

// ------------------------------------------------------ in float64 -------
// c of expert e; m and z as above.  Experts that are not finite rank last.
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

// Ranks a row anew; lane j returns the j-th expert.
__device__ __noinline__ int rank64(const Args& a, const float* row, int lane,
                                   float* max_logit, float* sum) {
  const int per = (a.E + 31) / 32, first = lane * per;
  bool bad = false;
  float m = -INFINITY;
  for (int e = lane; e < a.E; e += 32) {
    const float l = row[e];
    const bool ok = fabsf(l) <= FLT_MAX;
    bad |= !ok || (a.bias && !(fabsf(a.bias[e]) <= FLT_MAX));
    if (ok) m = fmaxf(m, l);
  }
  m = warp_max(m);
  double z = 0.0;
  if (!a.sigmoid) {
    for (int e = lane; e < a.E; e += 32)
      if (fabsf(row[e]) <= FLT_MAX)
        z += exp(static_cast<double>(row[e]) - static_cast<double>(m));
    z = warp_sum(z);
  }
  *max_logit = m;
  *sum = static_cast<float>(z);
  if (__any_sync(kAll, bad) && lane == 0 && a.status)
    atomicOr(a.status, MOE_DEV_NONFINITE);

  // the groups that take part, a lane for two of them
  unsigned long long keep = ~0ull;
  const int size = a.E / a.groups;
  if (a.top_groups < a.groups) {
    double total[2];
    for (int h = 0; h < 2; ++h) {
      const int g = h * 32 + lane;
      total[h] = -INFINITY;
      if (g >= a.groups) continue;
      double top[kMaxGroupTop];
      for (int j = 0; j < kMaxGroupTop; ++j) top[j] = -INFINITY;
      for (int e = g * size; e < (g + 1) * size; ++e) {
        double c = score64(a, row, e, m, z);
        for (int j = 0; j < a.group_top; ++j)
          if (c > top[j]) {
            const double t = top[j];
            top[j] = c;
            c = t;
          }
      }
      total[h] = top[0];
      for (int j = 1; j < a.group_top; ++j) total[h] += top[j];
    }
    int before[2] = {0, 0};
    for (int g = 0; g < a.groups; ++g) {
      const double t = __shfl_sync(kAll, g < 32 ? total[0] : total[1], g & 31);
      for (int h = 0; h < 2; ++h)
        if (t > total[h] || (t == total[h] && g < h * 32 + lane)) ++before[h];
    }
    keep = __ballot_sync(kAll, lane < a.groups && before[0] < a.top_groups);
    keep |= static_cast<unsigned long long>(__ballot_sync(
                kAll, 32 + lane < a.groups && before[1] < a.top_groups))
            << 32;
  }

  double c[32];
  uint32_t left = 0;  // this lane's experts that may be chosen yet
  for (int i = 0; i < per; ++i) {
    const int e = first + i;
    if (e < a.E && keep >> (e / size) & 1) {
      // without a bias the logits rank: their scores may round to the same
      c[i] = a.bias                       ? score64(a, row, e, m, z)
             : fabsf(row[e]) <= FLT_MAX ? static_cast<double>(row[e])
                                          : -INFINITY;
      left |= 1u << i;
    }
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY;
    int at = kMaxExperts;
    for (int i = 0; i < per; ++i)
      if (left >> i & 1 && (at == kMaxExperts || c[i] > best)) {
        best = c[i];
        at = first + i;
      }
    for (int o = 16; o > 0; o >>= 1) {
      const double other = __shfl_xor_sync(kAll, best, o);
      const int oat = __shfl_xor_sync(kAll, at, o);
      if (oat < kMaxExperts &&
          (at == kMaxExperts || other > best || (other == best && oat < at))) {
        best = other;
        at = oat;
      }
    }
    if (at >= first && at < first + per) left &= ~(1u << (at - first));
    if (lane == j) mine = at;
  }
  return mine;
}

// ------------------------------------------------------ in float32 -------
template <int EPL, int RANK>
__global__ void __launch_bounds__(kThreads) scores_kernel(const Args a) {
  // a row's candidates (c, expert), and for groups that are not whole lanes
  // its c
  __shared__ float cand_c[kWarps][32];
  __shared__ int cand_e[kWarps][32];
  extern __shared__ float row_c[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int size = a.E / a.groups;
  const bool select = a.top_groups < a.groups;
  // groups of whole lanes, a power of two of them
  const int lanes = size / EPL;
  const bool whole = size % EPL == 0 && (lanes & (lanes - 1)) == 0 &&
                     a.group_top <= 2;
  const int e0 = lane * EPL;
  const bool wide = EPL % 4 == 0 && a.E % 4 == 0 &&
                    (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
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
  for (long long t = blockIdx.x * static_cast<long long>(kWarps) + warp;
       t < a.T; t += gridDim.x * static_cast<long long>(kWarps)) {
    const float* row = a.logits + t * a.E;
    float c[EPL];
    bool again = most_bias == INFINITY;  // rank in float64
    bool loaded = false;
    if constexpr (EPL % 4 == 0) {
      if (wide) {
        loaded = true;
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
          float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          if (e0 + i < a.E)
            v = __ldg(reinterpret_cast<const float4*>(row + e0 + i));
          c[i] = v.x, c[i + 1] = v.y, c[i + 2] = v.z, c[i + 3] = v.w;
        }
      }
    }
    if (!loaded) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        c[i] = e0 + i < a.E ? __ldg(row + e0 + i) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      again |= e0 + i < a.E && !(fabsf(c[i]) <= FLT_MAX);

    // scores, and the most that a c may be off by
    float m = 0.0f, z = 1.0f, err = 0.0f;
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
    }
    if (RANK != kByLogit) {
      const float inv = RANK == kBySoftmax ? rcp_fast(z) : 1.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float s = RANK == kBySoftmax
                            ? c[i] * inv
                            : rcp_fast(1.0f + exp2_fast(-kLog2e * c[i]));
        c[i] = e0 + i < a.E ? s + bias[i] : -INFINITY;
      }
      // The sigmoid: 2^-22 of the exponential and what its argument's rounding
      // gives (a third of 2^-24), weighed by s (1 - s) <= 1/4, an ulp of the
      // reciprocal and half of one of the sum before it: below 2^-21.  The
      // softmax, of the largest score: its sum of up to 1024 terms is off by
      // 2^-22, by 17 2^-24 from the arguments (far terms: 10 bits of them at
      // most weigh) and by 37 2^-24 from adding: below 2^-18.  Adding the
      // bias: half an ulp.
      err = (RANK == kBySoftmax ? 3.8146973e-6f : 4.7683716e-7f) * inv +
            1.1920929e-7f * (inv + most_bias);
    }

    // this lane's two largest
    float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      m2 = fmaxf(m2, fminf(m1, c[i]));
      m1 = fmaxf(m1, c[i]);
    }
    if (select) {
      bool kept = false;
      if (whole) {
        float g1 = m1, g2 = m2;
        for (int o = 1; o < lanes; o <<= 1) {
          const float o1 = __shfl_xor_sync(kAll, g1, o);
          const float o2 = __shfl_xor_sync(kAll, g2, o);
          g2 = fmaxf(fminf(g1, o1), fmaxf(g2, o2));
          g1 = fmaxf(g1, o1);
        }
        const float total = a.group_top == 2 ? g1 + g2 : g1;
        const int mine = lane / lanes;
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
          const float other = __shfl_sync(kAll, total, g * lanes & 31);
          before += other > total || (other == total && g < mine);
        }
        const bool inside = e0 < a.E;
        kept = inside && before < a.top_groups;
        const float last = warp_min(kept ? total : INFINITY);
        const float next = warp_max(inside && !kept ? total : -INFINITY);
        // sums of n c are off by n errors, and adding them by n (n - 1) / 2
        if (RANK != kByLogit)
          again |= !(last - next > a.group_top * (a.group_top + 1) * err);
        if (!kept) {
          m1 = m2 = -INFINITY;
#pragma unroll
          for (int i = 0; i < EPL; ++i) c[i] = -INFINITY;
        }
      } else {
        // a lane a group (or two), over the row's c in shared memory
        float* rc = row_c + warp * (32 * EPL);
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
        const float last = warp_min(
            fminf(k0 ? total[0] : INFINITY, k1 ? total[1] : INFINITY));
        const float next =
            warp_max(fmaxf(lane < a.groups && !k0 ? total[0] : -INFINITY,
                           32 + lane < a.groups && !k1 ? total[1] : -INFINITY));
        if (RANK != kByLogit)
          again |= !(last - next > a.group_top * (a.group_top + 1) * err);
        const uint32_t low = __ballot_sync(kAll, k0);
        const uint32_t high = __ballot_sync(kAll, k1);
        m1 = m2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int g = (e0 + i) / size;
          if (g >= a.groups || !((g < 32 ? low >> g : high >> (g - 32)) & 1))
            c[i] = -INFINITY;
          m2 = fmaxf(m2, fminf(m1, c[i]));
          m1 = fmaxf(m1, c[i]);
        }
      }
    }

    // a threshold that at least k values reach, if the lanes' pairs hold k
    float bar = -INFINITY;
    uint32_t o1 = ordered(m1), o2 = ordered(m2);
    constexpr uint32_t kNone = 0x007fffffu;  // ordered(-infinity)
    for (int j = 0; j < a.k; ++j) {
      const uint32_t best = __reduce_max_sync(kAll, o1);
      bar = unordered(best);
      if (o1 == best) {
        o1 = o2;
        o2 = kNone;
      }
    }
    // values within twice the error of it stay, so that what is left out is
    // surely behind; a threshold of -infinity leaves nothing out
    bar = fmaxf(bar - 2.0f * err, -FLT_MAX);
    int n = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) n += c[i] >= bar;
    int at = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int below = __shfl_up_sync(kAll, at, o);
      if (lane >= o) at += below;
    }
    const int total = __shfl_sync(kAll, at, 31);
    at -= n;
    again |= total > 32 || total < a.k;

    int e = 0, rank = 32;
    float l = 0.0f;
    if (!__any_sync(kAll, again)) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (c[i] >= bar) {
          cand_c[warp][at] = c[i];
          cand_e[warp][at++] = e0 + i;
        }
      __syncwarp();
      const float v = lane < total ? cand_c[warp][lane] : -INFINITY;
      int before = 0;
      float gap = INFINITY;
      for (int j = 0; j < total; ++j) {
        const float other = __shfl_sync(kAll, v, j);
        before += other > v || (other == v && j < lane);
        if (RANK != kByLogit && j != lane) gap = fminf(gap, fabsf(other - v));
      }
      if (lane < total) {
        e = cand_e[warp][lane];
        rank = before;
        l = __ldg(row + e);
      }
      // nearer than the error allows, and before or among the k chosen
      if (RANK != kByLogit) again = rank <= a.k && gap <= 2.0f * err;
    }
    if (__any_sync(kAll, again)) {
      e = rank64(a, row, lane, &m, &z);
      rank = lane;
      l = lane < a.k ? row[e] : 0.0f;
      if (lane < a.k && a.bias && !(fabsf(a.bias[e]) <= FLT_MAX)) l = INFINITY;
    }
    const float w = weight(a, rank < a.k, l, m, z);
    if (rank < a.k) {
      a.idx[t * a.k + rank] = e;
      a.w[t * a.k + rank] = w;
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

// A chosen expert a lane.  With sigmoid scores the row is zero but for the
// chosen; with softmax scores lane i also has the i-th run of EPL experts.
template <bool SIGMOID>
__global__ void __launch_bounds__(kThreads) scores_backward_kernel(
    const BackArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool wide =
      a.E % 4 == 0 &&
      ((reinterpret_cast<uintptr_t>(a.logits) |
        reinterpret_cast<uintptr_t>(a.dlogits)) & 15) == 0;
  for (long long t = blockIdx.x * static_cast<long long>(kWarps) + warp;
       t < a.T; t += gridDim.x * static_cast<long long>(kWarps)) {
    const float* row = a.logits + t * a.E;
    float* out = a.dlogits + t * a.E;
    int e = -1 - lane;  // of no expert, and no other lane's
    float l = 0.0f, d = 0.0f;
    if (lane < a.k) {
      const int i = __ldg(a.idx + t * a.k + lane);
      d = __ldg(a.dw + t * a.k + lane);
      if (i >= 0 && i < a.E) {
        e = i;
        l = __ldg(row + e);
      }
    }
    const bool finite = e >= 0 && fabsf(l) <= FLT_MAX;
    float m = 0.0f, z = 1.0f;
    if (!SIGMOID) {
      m = -FLT_MAX;
      for (int i = lane; i < a.E; i += 32) {
        const float v = __ldg(row + i);
        if (fabsf(v) <= FLT_MAX) m = fmaxf(m, v);
      }
      m = warp_max(m);
      z = 0.0f;
      for (int i = lane; i < a.E; i += 32) {
        const float v = __ldg(row + i);
        if (fabsf(v) <= FLT_MAX) z += expf(v - m);
      }
      z = warp_sum(z);
    }
    // the weight over scale, as the forward has it
    const float top = a.renorm ? warp_max(finite ? l : -FLT_MAX) : 0.0f;
    float w = 0.0f;
    if (finite) {
      if (SIGMOID)
        w = expf(fminf(l, 0.0f) - (a.renorm ? fminf(top, 0.0f) : 0.0f)) /
            (1.0f + expf(-fabsf(l)));
      else
        w = a.renorm ? expf(l - top) : expf(l - m) / z;
    }
    if (a.renorm) {
      const float sum = warp_sum(w);
      w = sum > 0.0f ? w / sum : 0.0f;
    }
    float g = finite ? a.scale * d * w : 0.0f;
    if (a.renorm) g -= w * warp_sum(g);
    const float all = SIGMOID ? 0.0f : warp_sum(g);
    // an index that stands twice has the sum of both
    const uint32_t same = __match_any_sync(kAll, e);
    if (__any_sync(kAll, (same & (same - 1)) != 0)) {
      float sum = 0.0f;
      for (int j = 0; j < a.k; ++j) {
        const float other = __shfl_sync(kAll, g, j);
        if (same >> j & 1) sum += other;
      }
      g = sum;
    }
    if (wide) {
      for (int i = lane * 4; i < a.E; i += 128) {
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!SIGMOID) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(row + i));
          const float f = -all / z;
          o.x = fabsf(v.x) <= FLT_MAX ? f * expf(v.x - m) : 0.0f;
          o.y = fabsf(v.y) <= FLT_MAX ? f * expf(v.y - m) : 0.0f;
          o.z = fabsf(v.z) <= FLT_MAX ? f * expf(v.z - m) : 0.0f;
          o.w = fabsf(v.w) <= FLT_MAX ? f * expf(v.w - m) : 0.0f;
        }
        *reinterpret_cast<float4*>(out + i) = o;
      }
    } else {
      for (int i = lane; i < a.E; i += 32) {
        float o = 0.0f;
        if (!SIGMOID) {
          const float v = __ldg(row + i);
          if (fabsf(v) <= FLT_MAX) o = -all / z * expf(v - m);
        }
        out[i] = o;
      }
    }
    __syncwarp();  // the chosen are written over what other lanes wrote
    if (finite)
      out[e] = SIGMOID ? g * (1.0f / (1.0f + expf(l)))
                       : g - all / z * expf(l - m);
  }
}

unsigned token_grid(int T) {
  return static_cast<unsigned>(
      std::min<long long>((static_cast<long long>(T) + kWarps - 1) / kWarps,
                          1 << 14));
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

template <int EPL>
cudaError_t launch_epl(const Args& a, cudaStream_t s) {
  // the row's c, where groups are not whole lanes
  const int bytes =
      a.top_groups < a.groups ? kWarps * 32 * EPL * sizeof(float) : 0;
  const unsigned grid = token_grid(a.T);
  if (a.by_logit)
    scores_kernel<EPL, kByLogit><<<grid, kThreads, bytes, s>>>(a);
  else if (a.sigmoid)
    scores_kernel<EPL, kBySigmoid><<<grid, kThreads, bytes, s>>>(a);
  else
    scores_kernel<EPL, kBySoftmax><<<grid, kThreads, bytes, s>>>(a);
  return cudaGetLastError();
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
      !ok_ptr(dtopk_w, false) || !ok_ptr(dlogits, false))
    return MOE_ERR_INVALID_ARG;
  const BackArgs a = {logits, topk_idx, dtopk_w, dlogits, cfg->T, cfg->E,
                      cfg->k, opt->renorm != 0, opt->scale};
  const unsigned grid = token_grid(cfg->T);
  if (opt->score == MOE_SCORE_SIGMOID)
    scores_backward_kernel<true><<<grid, kThreads, 0, stream>>>(a);
  else
    scores_backward_kernel<false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
