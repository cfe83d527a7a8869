// Products of the routed rows with 4-bit expert weights (w4.cuh).
//
//   gate_up: h[r] = silu(x[r] Wg) * (x[r] Wu)      down: y[r] = h[r] Wd
//   W[k, n] = (code - zero) * scale, over groups of rows of W
//
// With few rows in a group the weights' bytes bound it, each read once.  So
// everything is arranged around that stream:
//
// * A warp works on two records (16 columns each): of the gate and the up
//   matrix, or two neighbours of the down matrix.  A matrix instruction
//   m16n8k16 takes 16 columns of weights as its 16-row operand and up to 8
//   rows of x as its 8 columns, so a batch of one token wastes no more than
//   idle lanes.
// * Next comes the arithmetic of expanding codes: logic and shifts run at 16
//   lanes a clock, so a tile of 64 rows of both records costs a scheduler 80
//   clocks of masks and byte shifts (see expand()), beside 72 of matrix
//   instructions and 64 of bf16 multiply-adds, against 172 at full bandwidth.
//   Measured instruction costs: 2 clocks for a mask, shift or bf16 pair, 9
//   for a matrix instruction, with little overlap of the two.
// * Weights go from HBM to a ring in shared memory by asynchronous 16-byte
//   copies, two steps of 256 rows ahead.  A lane reads back exactly what it
//   copied itself, so that ring needs no barrier.  (Bulk copies issued by one
//   warp were slower: about 1 KB each, 1300 us against 1000 us for the batch
//   of 64 below.)  CTAs are persistent and the ring runs on across work
//   items.
// * A work item is a record pair of NW warps (neighbouring columns, which
//   share the rows of x) with k split over KW warps, whose sums are added in
//   warp order, for one pass of up to 8 * NT rows.  Further rows of a group
//   are further items, whose weights come from L2.
//
// Measured, DeepSeek-V3-shaped experts (7168 x 2048, groups of 128): one
// token 44.7 us (8 experts, 182 MB: 4.1 TB/s; the launches and the tail of
// 6.7 items an SM are what it loses); 16 tokens over 32
// experts 142 us (5.1 TB/s; the copies alone 119 us, the arithmetic alone 145
// us); 64 tokens, Zipf, 650 us (5.0 TB/s).  Llama4-Maverick-shaped, 16 tokens
// one expert each, groups of 32 with zero points: 186 to 208 us, with where the
// weights lie in memory (6.1 to 5.4 TB/s).
//
// float32 rows use the same instructions: a float is the exact sum of three
// bf16 numbers (8 bits of its significand each), so three products with the
// exact weights give float32 accuracy.  A matrix instruction truncates what it
// adds to, so the leading parts are summed apart from the others, over at most
// 64 rows of W: their products are short, most of their sums exact, and what
// the sums of the small parts lose is 2^-8 of what it would be in one sum.
// (256 x 512, groups of 128: y is 1e-7 off, normwise; in one sum it was 1.4e-6
// and always towards zero, for 0 to 3% less time.)  Every block of 16 columns
// splits the rows again, and that bounds them: one token of the 7168 x 2048
// experts 99 us, 64 tokens of 32 experts (16 rows each) 900 us.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>

#include "launch.cuh"
#include "tc_common.cuh"
#include "w4.cuh"

namespace moe {
namespace w4 {

using launch::Device;

// Products of one row type (gmm_w4_bf16.cu, gmm_w4_f32.cu): dual is gate_up.
struct GmmArgs;
cudaError_t launch_gmm_w4_bf16(bool dual, const GmmArgs& a, int tokens,
                               cudaStream_t s);
cudaError_t launch_gmm_w4_f32(bool dual, const GmmArgs& a, int tokens,
                              cudaStream_t s);
// Groups of many bf16 rows (gmm_w4_tc.cu).
cudaError_t launch_gmm_w4_tc(bool dual, GmmArgs a, cudaStream_t s);

constexpr int kTiles = kStepK / kTileK;  // tiles of a step
constexpr int kUnit = 2;                 // tiles copied and waited for at once
constexpr int kUnits = kTiles / kUnit;
constexpr int kXSlots = 3;               // steps of x (and scales) held
constexpr int kRing = 2 * kTiles;        // tiles of codes held: two steps

struct GmmArgs {
  const char* x;
  const int32_t *offsets, *map;
  const char *w0, *w1;
  void* out;
  int32_t* status;
  Layout l;
  int n_experts, n_groups, rows;
  int chunk;   // rows of a group that one work item takes
  int chunks;  // at most so many in all
  int x_rows;  // rows of x that a slot holds: those of one pass
  bool early;  // may start before the kernel that writes x has ended
};

// ---------------------------------------------------------------- PTX ----
using tc::smem_u32;
// 16 bytes, zeros where `in` is false (then src is not read).
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src,
                                               bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
// D = C + A B: A 16 weight columns x 16 k, B 16 k x 8 rows of x.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4],
                                    uint32_t b0, uint32_t b1,
                                    const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1),
        "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// a * b + c on bf16 pairs.
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// Powers of two as bf16 pairs.
constexpr uint32_t kPow127 = 0x7f007f00u, kPow123 = 0x7d007d00u;

// The operand registers of one word of codes: (code - zero) / 64 as bf16
// pairs, exactly.  The low eight bits of a bf16 whose other bits are zero
// are a whole number times 2^-133 (a subnormal, or the first binade, which
// continues them), so a masked code needs no shift within its byte, and the
// multiplication that scales it subtracts the zero as well: z holds -zero/64
// of columns c and c + 8.
__device__ __forceinline__ void expand(uint32_t w, const uint32_t (&z)[2],
                                       uint32_t (&a)[4]) {
  const uint32_t v = w >> 8;
  a[0] = fma2(w & 0x000f000fu, kPow127, z[0]);
  a[1] = fma2(w & 0x00f000f0u, kPow123, z[1]);
  a[2] = fma2(v & 0x000f000fu, kPow127, z[0]);
  a[3] = fma2(v & 0x00f000f0u, kPow123, z[1]);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16(v);
}

// The chunks of rows of the groups that have rows and an expert, in order:
// (group, first row); their number.
template <int WARPS, typename A>
__device__ int find_chunks(const A& a, int2* chunks) {
  __shared__ int count[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int total = 0;
  for (int g0 = 0; g0 < a.n_groups; g0 += WARPS * 32) {
    const int g = g0 + threadIdx.x;
    int n = 0, row = 0;
    if (g < a.n_groups) {
      row = max(0, a.offsets[g]);
      const int rows = min(a.rows, a.offsets[g + 1]) - row;
      if (rows > 0) n = (rows - 1) / a.chunk + 1;
      const int ex = n > 0 && a.map ? a.map[g] : g < a.n_experts ? g : -1;
      if (n > 0 && (ex < 0 || ex >= a.n_experts)) {
        n = 0;
        if (blockIdx.x == 0 && a.status)
          atomicOr(a.status, MOE_DEV_BAD_INDEX);
      }
    }
    int upto = n;  // of this warp's groups, this one's included
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int below = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += below;
    }
    if (lane == 31) count[warp] = upto;
    __syncthreads();
    int at = total + upto - n;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) at += count[w];
      total += count[w];
    }
    // offsets that overlap could make more than there is room for
    for (int i = 0; i < n && at + i < a.chunks; ++i)
      chunks[at + i] = make_int2(g, row + i * a.chunk);
    __syncthreads();
  }
  return min(total, a.chunks);
}
// The end of the chunk's rows.
template <typename A>
__device__ __forceinline__ int chunk_end(const A& a, int2 c) {
  const int end = min(a.rows, a.offsets[c.x + 1]);
  return end - c.y > a.chunk ? c.y + a.chunk : end;
}

// The operands of 32 k of eight rows of x: P parts, two instructions each.
// lane_at() is where a lane reads, from the start of its row's 32 k; the
// lane's row is row(lane) of the eight.
template <typename T>
struct Rows;
template <>
struct Rows<__nv_bfloat16> {
  static constexpr int P = 1;
  static constexpr int kPad = 16;  // rows 16 bytes apart mod 128: no conflict
  static __device__ __forceinline__ int row(int lane) { return lane & 7; }
  static __device__ __forceinline__ int lane_at(int lane) {
    return lane / 8 * 16;
  }
  uint32_t q[4];
  __device__ __forceinline__ void load(uint32_t a) {
    asm volatile(
        "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
        : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3])
        : "r"(a)
        : "memory");
  }
  __device__ __forceinline__ void part(int, uint32_t (&b)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = q[i];
  }
};
template <>
struct Rows<float> {
  static constexpr int P = 3;
  static constexpr int kPad = 32;  // four rows of 32 bytes side by side
  static __device__ __forceinline__ int row(int lane) { return lane >> 2; }
  static __device__ __forceinline__ int lane_at(int lane) {
    return (lane & 3) * 8;
  }
  float f[8];
  __device__ __forceinline__ void load(uint32_t a) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                   : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
                   : "r"(a + 32 * i)
                   : "memory");
  }
  // Takes the leading 8 bits of what is left, by truncation: no part
  // overflows and the rest is exact.  Nothing is left of an infinity.
  __device__ __forceinline__ void part(int, uint32_t (&b)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float& v = f[2 * i + j];
        h[j] = __float_as_uint(v) & 0xffff0000u;
        const float top = __uint_as_float(h[j]);
        v = v == top ? 0.0f : v - top;
      }
      b[i] = __byte_perm(h[0], h[1], 0x7632);
    }
  }
};

// Where a warp stands in its sequence of steps.
struct Cursor {
  int item, row, r1, step;  // r1: end of the group's rows
};

template <typename T, bool DUAL, int NW, int KW, int NT, int G, bool Z>
struct Kernel {
  static constexpr int kWarps = NW * KW;
  static constexpr int kThreads = kWarps * 32;
  static constexpr bool kShareX = NW > 1;  // else each warp copies its own k
  static constexpr int kRows = 8 * NT;
  static constexpr int kStepBytes = kStepK * sizeof(T);
  static constexpr int kPitch = kStepBytes + Rows<T>::kPad;
  static constexpr int E = kStepK / G;  // groups of a step
  static constexpr int kScaleRec = 8 * E * (Z ? 6 : 4);  // of a step
  static constexpr int kChunk = kTiles * kTileBytes + kScaleRec;
  static constexpr int kTilePair = 2 * kTileBytes;
  // CTAs an SM has registers for.  A fifth CTA of four warps (96 registers a
  // thread) takes one bf16 token from 47.1 to 44.7 us; float32 rows, whose
  // three parts need the registers, from 49 to 51 us.
  static constexpr int kPerSm = kWarps == 8 ? 2 : sizeof(T) == 2 ? 5 : 4;
  // columns of an item
  static constexpr int kCols = DUAL ? NW * kTileN : 2 * NW * kTileN;
  static_assert(!kShareX || KW == 1, "x is shared by warps of the same k");

  // Shared memory: codes [warp][kRing][2][512], x [slot](or [slot][warp])
  // [rows][pitch], scales and zeros [slot][warp][2], sums, active groups.
  struct Smem {
    int x, x_slot, scales, sums, groups, total;
  };
  __host__ __device__ static constexpr Smem smem(int x_rows, int chunks) {
    Smem m = {};
    m.x = kWarps * kRing * kTilePair;
    m.x_slot = (kShareX ? 1 : kWarps) * x_rows * kPitch;
    m.scales = m.x + kXSlots * m.x_slot;
    m.sums = m.scales + kXSlots * kWarps * 2 * kScaleRec;
    m.groups = m.sums + (KW > 1 ? kWarps * 2 * x_rows * kTileN * 4 : 0);
    m.total = m.groups + 8 * chunks + 16;
    return m;
  }

  __device__ static void run(const GmmArgs& a) {
    extern __shared__ __align__(128) char base[];
    const Layout l = a.l;
    const Smem m = smem(a.x_rows, a.chunks);
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int nw = warp % NW, kw = warp / NW;
    const int c = lane >> 2, t = lane & 3;
    const int tiles_k = l.tiles_k(), n_steps = l.steps();
    const uint32_t sb = smem_u32(base);
    int2* chunks = reinterpret_cast<int2*>(base + m.groups);
    launch::let_next_start();
    const int n_chunks = find_chunks<kWarps>(a, chunks);  // a barrier within
    const int blocks = (l.N + kCols - 1) / kCols;
    const int n_items = n_chunks * blocks;

    // --- the copying side, two steps ahead: this lane's place in the
    // warp's records of the cursor's step, and in the rows of x
    Cursor in = {};
    const char *p0 = nullptr, *p1 = nullptr, *xp = nullptr;
    int left = 0;  // tiles of the cursor's step and after, 0 past the end
    const long long row_bytes = static_cast<long long>(l.K) * sizeof(T);
    // rows side by side in a warp's copy, and the lane's word of its row
    constexpr int kWords = kStepBytes / 16;
    constexpr int kSide = kWords < 32 ? 32 / kWords : 1;
    const int x_first = (kShareX ? warp * kSide : 0) + lane * kSide / 32;
    constexpr int kRowStride = (kShareX ? kWarps : 1) * kSide;
    const int x_word = lane % (32 / kSide) * 16;
    const uint32_t x_dst = sb + m.x +
                           (kShareX ? 0 : warp * a.x_rows * kPitch) +
                           x_first * kPitch + x_word;
    const auto rewind = [&] {  // to the first step, rows from in.row on
      in.step = kw;
      left = tiles_k - kw * kTiles;
      xp = a.x + (in.row + x_first) * row_bytes + kw * kStepBytes + x_word;
    };
    const auto enter = [&] {  // the item's group and records
      const int2 chunk = chunks[in.item / blocks];
      const int nb = in.item % blocks;
      const int ex = a.map ? a.map[chunk.x] : chunk.x;
      in.row = chunk.y;
      in.r1 = chunk_end(a, chunk);
      // a record past the last one is the last again: its columns are not
      // written
      const int rec = DUAL ? nb * NW + nw : 2 * (nb * NW + nw);
      const int last = l.tiles_n() - 1;
      const long long mat = ex * l.matrix(), len = l.record();
      const int at = kw * kChunk + lane * 16;
      p0 = a.w0 + mat + min(rec, last) * len + at;
      p1 = DUAL ? a.w1 + mat + min(rec, last) * len + at
                : a.w0 + mat + min(rec + 1, last) * len + at;
      rewind();
    };
    const auto advance = [&] {
      in.step += KW;
      left -= KW * kTiles;
      p0 += KW * kChunk;
      p1 += KW * kChunk;
      xp += KW * kStepBytes;
      if (left > 0) return;
      in.row += a.x_rows;
      if (in.row < in.r1) {  // the group's next rows: the same weights
        const long long back =
            static_cast<long long>((in.step - kw) / KW) * (KW * kChunk);
        p0 -= back;
        p1 -= back;
        rewind();
      } else {
        in.item += gridDim.x;
        if (in.item < n_items) enter();
      }
    };
    const uint32_t codes = sb + warp * (kRing * kTilePair) + lane * 16;
    const uint32_t sc0 = sb + m.scales + warp * 2 * kScaleRec;
    // Tiles first.. of the cursor's step into slot `half` (of two).
    const auto copy_codes = [&](int half, int first) {
      const uint32_t dst = codes + (half * kTiles + first) * kTilePair;
      const auto copy_tile = [&](int i) {
        copy16(dst + i * kTilePair, p0 + (first + i) * kTileBytes);
        copy16(dst + i * kTilePair + kTileBytes,
               p1 + (first + i) * kTileBytes);
      };
      if (left >= first + kUnit) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) copy_tile(i);
      } else if (left > first) {
        copy_tile(0);
      }
    };
    // The step's scales and rows of x into slot xs (of three).
    const auto copy_scales = [&](int xs) {
      if (left > 0 && lane * 16 < kScaleRec) {
        const int at = min(left, kTiles) * kTileBytes;
        const uint32_t d = sc0 + xs * kWarps * 2 * kScaleRec + lane * 16;
        copy16(d, p0 + at);
        copy16(d + kScaleRec, p1 + at);
      }
    };
    const auto copy_rows = [&](int xs) {
      if (left <= 0) return;
      const int rows = min(a.x_rows, in.r1 - in.row) - x_first;
      const long long rest =  // of the rows from this lane's place on
          row_bytes - static_cast<long long>(in.step) * kStepBytes - x_word;
      const uint32_t d = x_dst + xs * m.x_slot;
      // a warp that copies for itself has one row or few
#pragma unroll(kShareX ? kRows / kRowStride : 1)
      for (int r = 0; r < (kShareX ? kRows : rows); r += kRowStride)
        if (!kShareX || r < rows)
#pragma unroll
          for (int w = 0; w < kWords; w += 32)
            copy16_or_zero(d + r * kPitch + w * 16,
                           xp + r * row_bytes + w * 16, w * 16 < rest);
    };
    const auto copy_unit = [&](int half, int xs, int first) {
      copy_codes(half, first);
      if (first == 0) {
        copy_scales(xs);
        copy_rows(xs);
      }
      copies_commit();
    };

    // The first two steps: weights first, then, once the kernel before this
    // one has written them, the rows.
    const auto begin = [&](bool weights) {
      in.item = blockIdx.x;
      left = 0;
      if (in.item < n_items && kw < n_steps) enter();
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        if (weights) {
          for (int u = 0; u < kUnits; ++u) copy_codes(s, u * kUnit);
          copy_scales(s);
        } else {
          copy_rows(s);
        }
        if (left > 0) advance();
      }
    };
    begin(true);
    launch::wait_for_previous();
    begin(false);
#pragma unroll
    for (int u = 0; u < 2 * kUnits; ++u) copies_commit();

    // --- the computing side
    int half = 0, xs = 0;  // the slots of the step
    uint32_t x_row[NT];  // this lane's row of each eight
#pragma unroll
    for (int b = 0; b < NT; ++b)
      x_row[b] = sb + m.x + (kShareX ? 0 : warp * a.x_rows * kPitch) +
                 Rows<T>::lane_at(lane) +
                 min(8 * b + Rows<T>::row(lane), a.x_rows - 1) * kPitch;
#pragma unroll 1
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
      const int2 chunk = chunks[item / blocks];
      const int r1 = chunk_end(a, chunk);
#pragma unroll 1
      for (int row = chunk.y; row < r1; row += a.x_rows) {
        const int rows = min(a.x_rows, r1 - row);
        float acc[2][NT][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][b][i] = 0.0f;
#pragma unroll 1
        for (int step = kw; step < n_steps; step += KW) {
          const int tiles = tiles_k - step * kTiles;
          const uint32_t x0 = xs * m.x_slot;
          const uint32_t sc =
              sc0 + xs * kWarps * 2 * kScaleRec + c * 4 * E;
          const uint32_t w = codes + half * kTiles * kTilePair;
          const int next = xs == 0 ? kXSlots - 1 : xs - 1;  // two on
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            copies_wait<2 * kUnits - 1>();
            if (u == 0) {
              if (kShareX)
                __syncthreads();
              else
                __syncwarp();
            }
            if (tiles >= (u + 1) * kUnit)
              multiply<kUnit>(acc, rows, w + u * kUnit * kTilePair,
                              x_row, x0, sc, u * kUnit, c);
            else if (tiles > u * kUnit)
              multiply<1>(acc, rows, w + u * kUnit * kTilePair, x_row,
                          x0, sc, u * kUnit, c);
            // the slot's next tiles: this lane has read what they overwrite
            copy_unit(half, next, u * kUnit);
          }
          if (left > 0) advance();
          half ^= 1;
          xs = xs == kXSlots - 1 ? 0 : xs + 1;
        }
        finish(a, m, acc, row, (item % blocks) * kCols, rows, base, warp, nw,
               c, t);
      }
    }
    copies_wait<0>();
  }

  // TILES tiles of both records, from tile `first` of the step on, times the
  // rows of x.
  template <int TILES>
  __device__ static __forceinline__ void multiply(
      float (&acc)[2][NT][4], int rows, uint32_t codes,
      const uint32_t (&x_row)[NT], uint32_t x0, uint32_t sc, int first,
      int c) {
    uint32_t w[TILES][2][4];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 q = lds16(codes + i * kTilePair + r * kTileBytes);
        w[i][r][0] = q.x, w[i][r][1] = q.y, w[i][r][2] = q.z;
        w[i][r][3] = q.w;
      }
    // of the leading part of x, and of the others
    constexpr int kSums = Rows<T>::P > 1 ? 2 : 1;
    constexpr int kSumK = kSums > 1 && G > kTileK ? kTileK : G;  // rows in one
    float part[kSums][2][NT][4], s[2][2];
    uint32_t zero[2][2];
    constexpr int kHalves = 2 * TILES;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int k = first * kTileK + 32 * h;
      if (h == 0 || k % G == 0) {  // a group begins
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t pair = lds4(sc + r * kScaleRec + k / G * 4);
          s[r][0] = __uint_as_float(pair << 16);
          s[r][1] = __uint_as_float(pair & 0xffff0000u);
          zero[r][0] = zero[r][1] = 0xbe00be00u;  // -8/64
          if (Z) {
            const uint32_t z =
                lds2(sc + r * kScaleRec + (32 - 2 * c) * E + k / G * 2);
            zero[r][0] = fma2(__byte_perm(z, 0, 0x4040), kPow127 | 0x80008000u, 0);
            zero[r][1] = fma2(__byte_perm(z, 0, 0x4141), kPow127 | 0x80008000u, 0);
          }
        }
      }
      if (h == 0 || k % kSumK == 0) {
#pragma unroll
        for (int q = 0; q < kSums; ++q)
#pragma unroll
          for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              part[q][0][b][i] = part[q][1][b][i] = 0.0f;
      }
      uint32_t op[2][2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          expand(w[h / 2][r][h % 2 * 2 + i], zero[r], op[r][i]);
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        if (NT > 1 && 8 * b >= rows) break;
        Rows<T> v;
        v.load(x_row[b] + x0 + first * kTileK * static_cast<int>(sizeof(T)) +
               h * 32 * static_cast<int>(sizeof(T)));
#pragma unroll
        for (int p = 0; p < Rows<T>::P; ++p) {
          uint32_t o[4];
          v.part(p, o);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float(&d)[4] = part[p == 0 ? 0 : kSums - 1][r][b];
              mma(d, op[r][i], o[2 * i], o[2 * i + 1], d);
            }
        }
        if (h == kHalves - 1 || (k + 32) % kSumK == 0) {  // a sum ends
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v = part[0][r][b][i];
              if (kSums > 1) v += part[kSums - 1][r][b][i];
              acc[r][b][i] = fmaf(s[r][i >> 1], v, acc[r][b][i]);
            }
        }
      }
    }
  }

  // Adds the warps' sums over k and writes the rows' columns.
  __device__ static __forceinline__ void finish(
      const GmmArgs& a, const Smem& m, const float (&acc)[2][NT][4], int row,
      int n0, int rows, char* base, int warp, int nw, int c, int t) {
    T* out = static_cast<T*>(a.out);
    if (KW == 1) {
      // a lane holds rows 2t and 2t + 1 of each 8, columns c and c + 8
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * b + 2 * t + (i & 1);
          if (r >= rows) continue;
          const int col = c + 8 * (i >> 1);
          T* o = out + static_cast<long long>(row + r) * a.l.N;
          if (DUAL) {
            const int n = n0 + nw * kTileN + col;
            if (n < a.l.N) put(o + n, swiglu(acc[0][b][i], acc[1][b][i]));
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int n = n0 + (2 * nw + h) * kTileN + col;
              if (n < a.l.N) put(o + n, 64.0f * acc[h][b][i]);
            }
          }
        }
      return;
    }
    float* sums = reinterpret_cast<float*>(base + m.sums);
    const int rec_floats = a.x_rows * kTileN;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * b + 2 * t + (i & 1);
          if (r < rows)
            sums[(warp * 2 + h) * rec_floats + r * kTileN + c +
                 8 * (i >> 1)] = acc[h][b][i];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * kCols; i += kThreads) {
      const int r = i / kCols, rec = i % kCols / kTileN, col = i % kTileN;
      const int w = DUAL ? rec : rec >> 1, h = DUAL ? 0 : rec & 1;
      const int n = n0 + i % kCols;
      if (n >= a.l.N) continue;
      float v = 0.0f, u = 0.0f;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const float* p = sums + ((k * NW + w) * 2 + h) * rec_floats +
                         r * kTileN + col;
        v += *p;
        if (DUAL) u += p[rec_floats];
      }
      put(out + static_cast<long long>(row + r) * a.l.N + n,
          DUAL ? swiglu(v, u) : 64.0f * v);
    }
    __syncthreads();
  }

  // of sums that are 1/64 of the products
  __device__ static __forceinline__ float swiglu(float g, float u) {
    g *= 64.0f;
    u *= 64.0f;
    return g / (1.0f + expf(-g)) * u;
  }
};

template <typename T, bool DUAL, int NW, int KW, int NT, int G, bool Z>
__global__ void __launch_bounds__(
    NW* KW * 32, Kernel<T, DUAL, NW, KW, NT, G, Z>::kPerSm)
    gmm_w4_kernel(const GmmArgs a) {
  Kernel<T, DUAL, NW, KW, NT, G, Z>::run(a);
}

// Chunks of as few passes of `rows` rows as leave at most kMaxSplits more
// than there are groups.  CTAs that take chunks of one group at the same time
// share its weights in L2.
constexpr int kMaxSplits = 512;
constexpr int kMaxChunks = kMaxExperts + kMaxSplits;
// Dynamic shared memory that every CTA may have: 227 KB, less 1 KB for the
// kernels' own static arrays.
constexpr int kMaxShared = 226 * 1024;
inline void set_chunk(GmmArgs* a, int rows) {
  const long long most = static_cast<long long>(rows) * kMaxSplits;
  a->chunk = rows * static_cast<int>((a->rows + most - 1) / most);
  a->chunks = std::min(a->n_groups, a->rows) + a->rows / a->chunk;
}

template <typename T, bool DUAL, int NW, int KW, int NT, int G, bool Z>
cudaError_t launch_one(GmmArgs a, int tokens, const Device& d,
                       cudaStream_t s) {
  using Ker = Kernel<T, DUAL, NW, KW, NT, G, Z>;
  // routing gives a group at most one row of each token
  a.x_rows = std::max(1, std::min(Ker::kRows, tokens));
  set_chunk(&a, a.x_rows);
  static_assert(Ker::smem(Ker::kRows, kMaxChunks).total <= kMaxShared,
                "any call's shared memory fits a CTA");
  const int bytes = Ker::smem(a.x_rows, a.chunks).total;
  constexpr auto kernel = gmm_w4_kernel<T, DUAL, NW, KW, NT, G, Z>;
  const cudaError_t e = launch::allow_shared<kernel>(d);
  if (e != cudaSuccess) return e;
  const int per_sm = std::min(Ker::kPerSm, d.smem_sm / (bytes + 1024));
  const long long items =
      static_cast<long long>((a.l.N + Ker::kCols - 1) / Ker::kCols) *
      a.chunks;
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>(items, static_cast<long long>(per_sm) * d.sms));
  if (a.early)
    return launch::overlapping(kernel, grid, Ker::kThreads, bytes, s, a);
  kernel<<<grid, Ker::kThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool DUAL, int G, bool Z>
cudaError_t launch_shape(const GmmArgs& a, int tokens, cudaStream_t s) {
  Device d;
  const cudaError_t e = launch::device(&d);
  if (e != cudaSuccess) return e;
  // Work items of 128 columns (of both matrices, or 256 of the one), if rows
  // spread evenly over the groups and a pass takes `rows` of them.
  const long long groups = std::min(a.n_groups, a.rows);
  const long long each = (a.rows + groups - 1) / groups;
  const auto items = [&](int rows) {
    return groups * ((a.l.N + (DUAL ? 127 : 255)) / (DUAL ? 128 : 256)) *
           ((each + rows - 1) / rows);
  };
  // A pass takes 8 rows (NT = 1), 16 (NT = 2) or 48 (tcgen05).  32 groups of
  // 7168 x 2048 with 16 rows each: 243 us on NT = 2, 324 us on tcgen05; 24
  // rows: 332 and 333 us; 32 rows: 421 and 339 us; 64 rows: 748 and 602 us.
  const bool many = sizeof(T) == 2 && a.rows > 20 * groups;
  // Too few items for the SMs: 16 columns an item, and k over four warps.
  // 33 float32 tokens, three of 7 experts each, 1412 x 1004: 49 us, and 76 us
  // in items of 128 columns; 4 tokens of 256 experts 132 us, and 158 us with k
  // over eight warps.
  const long long wide = items(many ? 48 : a.rows <= 4 * groups ? 8 : 16);
  if (wide < (tokens <= 8 ? 4 : 1) * static_cast<long long>(d.sms))
    return launch_one<T, DUAL, 1, 4, 1, G, Z>(a, tokens, d, s);
  if (many) return launch_gmm_w4_tc(DUAL, a, s);
  if (a.rows <= 4 * groups)
    return launch_one<T, DUAL, 8, 1, 1, G, Z>(a, tokens, d, s);
  return launch_one<T, DUAL, 8, 1, 2, G, Z>(a, tokens, d, s);
}

// The products of one row type: what gmm_w4_bf16.cu and gmm_w4_f32.cu each
// instantiate, apart so that they compile side by side.
template <typename T, bool DUAL>
cudaError_t launch_rows(const GmmArgs& a, int tokens, cudaStream_t s) {
#define MOE_W4_CASE(GROUP)                                        \
  if (a.l.group == GROUP)                                         \
    return a.l.zeros                                              \
               ? launch_shape<T, DUAL, GROUP, true>(a, tokens, s) \
               : launch_shape<T, DUAL, GROUP, false>(a, tokens, s)
  MOE_W4_CASE(32);
  MOE_W4_CASE(64);
  MOE_W4_CASE(128);
#undef MOE_W4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace w4
}  // namespace moe
