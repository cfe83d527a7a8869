// Products of the routed rows with 4-bit expert weights (w4.cuh).
//
//   gate_up: h[r] = silu(x[r] Wg) * (x[r] Wu)      down: y[r] = h[r] Wd
//   W[k, n] = (code - zero) * scale, over groups of rows of W
//
// What bounds it is the weights' bytes, each read once, as long as a group
// has few rows.  So everything is arranged around that stream:
//
// * A warp works on two records (16 columns each): of the gate and the up
//   matrix, or two neighbours of the down matrix.  A matrix instruction
//   m16n8k16 takes 16 columns of weights as its 16-row operand and up to 8
//   rows of x as its 8 columns, so a batch of one token wastes no more than
//   idle lanes.
// * Issue slots come next: 1 KB of codes (one tile of both records) has 172
//   at full bandwidth.  A code masked into bits 3..6 of a bf16 128 is
//   8 * (16 + code), one rotation and one logic operation for two of them,
//   and nothing is subtracted from it: the sums start from those of the
//   constant operand -8 * (16 + zero), four more matrix instructions.  That
//   sum is at most 31/7.5 times as large as the one it stands for, so
//   float32 loses about two bits of its 24.  The scale multiplies the
//   partial sum of each 32 or 64 rows of W, the 1/8 the final one.
// * Weights go from HBM to a ring in shared memory by asynchronous 16-byte
//   copies, two steps of 256 rows ahead.  A lane reads back exactly what it
//   copied itself, so that ring needs no barrier.  CTAs are persistent, one
//   or two an SM, and the ring runs on across work items.
// * A work item is a record pair of NW warps (neighbouring columns, which
//   share the rows of x) with k split over KW warps, whose sums are added in
//   warp order.  Many items: NW = 8 or 16; a few tokens leave few groups and
//   few items, then NW = 1, KW = 8.
// * More rows than 8 * NT of a group are further passes over its weights,
//   which then come from L2.
//
// float32 rows use the same instructions: a float is the exact sum of three
// bf16 numbers (8 bits of its significand each), so three products with the
// exact weights give float32 accuracy.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>

#include "w4.cuh"

namespace moe {
namespace w4 {

// Products of one row type (gmm_w4_bf16.cu, gmm_w4_f32.cu): dual is gate_up.
struct GmmArgs;
cudaError_t launch_gmm_w4_bf16(bool dual, const GmmArgs& a, int tokens,
                               cudaStream_t s);
cudaError_t launch_gmm_w4_f32(bool dual, const GmmArgs& a, int tokens,
                              cudaStream_t s);

constexpr int kTiles = kStepK / kTileK;  // tiles of a step
constexpr int kXSlots = 3;               // steps of x (and scales) held
constexpr int kRing = 2 * kTiles;        // tiles of codes in flight

struct GmmArgs {
  const char* x;
  const int32_t *offsets, *map;
  const char *w0, *w1;
  void* out;
  int32_t* status;
  Layout l;
  int n_experts, n_groups, rows;
  int x_rows;  // rows of x that a slot holds: those of one pass
};

// ---------------------------------------------------------------- PTX ----
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
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
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst),
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

// The operand registers of one word of codes: 8 * (16 + code) as bf16
// pairs, exactly.  `one` holds two bf16 128, from shared memory: a known
// constant would be moved into a register again for every use.
__device__ __forceinline__ void expand(uint32_t w, uint32_t one,
                                       uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = (__funnelshift_r(w, w, 4 * i) & 0x00780078u) | one;
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16(v);
}

// The operands of eight k of one row of x: P parts, two instructions each.
template <typename T>
struct Rows;
template <>
struct Rows<__nv_bfloat16> {
  static constexpr int P = 1;
  static constexpr int kLaneBytes = 16;
  static constexpr int kPad = 64;  // rows 64 bytes apart mod 128: no conflict
  uint4 q;
  __device__ __forceinline__ void load(uint32_t a) { q = lds16(a); }
  __device__ __forceinline__ void part(int, uint32_t (&b)[4]) const {
    b[0] = q.x, b[1] = q.y, b[2] = q.z, b[3] = q.w;
  }
};
template <>
struct Rows<float> {
  static constexpr int P = 3;
  static constexpr int kLaneBytes = 32;
  static constexpr int kPad = 16;
  float f[8];
  __device__ __forceinline__ void load(uint32_t a) {
    const uint4 u = lds16(a), v = lds16(a + 16);
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
    f[4] = __uint_as_float(v.x), f[5] = __uint_as_float(v.y);
    f[6] = __uint_as_float(v.z), f[7] = __uint_as_float(v.w);
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
  // columns of an item
  static constexpr int kCols = DUAL ? NW * kTileN : 2 * NW * kTileN;
  static_assert(!kShareX || KW == 1, "x is shared by warps of the same k");

  // Shared memory: codes [warp][kRing][2][512], x [slot](or [slot][warp])
  // [rows][pitch], scales and zeros [slot][warp][2], sums, active groups.
  struct Smem {
    int x, x_slot, scales, sums, groups, total;
  };
  __host__ __device__ static Smem smem(int x_rows, int n_groups) {
    Smem m;
    m.x = kWarps * kRing * kTilePair;
    m.x_slot = (kShareX ? 1 : kWarps) * x_rows * kPitch;
    m.scales = m.x + kXSlots * m.x_slot;
    m.sums = m.scales + kXSlots * kWarps * 2 * kScaleRec;
    m.groups = m.sums + (KW > 1 ? kWarps * 2 * kRows * kTileN * 4 : 0);
    m.total = m.groups + 4 * n_groups + 16;
    return m;
  }

  __device__ static void run(const GmmArgs& a) {
    extern __shared__ __align__(128) char base[];
    const Layout l = a.l;
    const Smem m = smem(a.x_rows, a.n_groups);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nw = warp % NW, kw = warp / NW;
    const int c = lane >> 2, t = lane & 3;
    const int tiles_k = l.tiles_k(), n_steps = l.steps();
    const uint32_t sb = smem_u32(base);
    int32_t* active = reinterpret_cast<int32_t*>(base + m.groups);
    __shared__ uint32_t constant;
    if (threadIdx.x == 0) constant = 0x43004300u;
    const int n_active = find_active(a, active);  // a barrier within
    const uint32_t one = lds4(smem_u32(&constant));
    const int blocks = (l.N + kCols - 1) / kCols;
    const int n_items = n_active * blocks;

    // --- the copying side, two steps ahead: this lane's place in the
    // warp's records of the cursor's step, and in the rows of x
    Cursor in = {};
    const char *p0 = nullptr, *p1 = nullptr, *xp = nullptr;
    int left = 0;  // tiles of the cursor's step and after, 0 past the end
    const long long row_bytes = static_cast<long long>(l.K) * sizeof(T);
    // a lane copies the words x_lane, x_lane + 32, ... of row x_first, ...
    constexpr int kWords = kStepBytes / 16;
    const int x_first = kShareX ? warp : 0;
    constexpr int kRowStride = kShareX ? kWarps : 1;
    const uint32_t x_dst = sb + m.x +
                           (kShareX ? 0 : warp * a.x_rows * kPitch) +
                           x_first * kPitch + lane * 16;
    const auto rewind = [&] {  // to the first step, rows from in.row on
      in.step = kw;
      left = tiles_k - kw * kTiles;
      xp = a.x + (in.row + x_first) * row_bytes + kw * kStepBytes + lane * 16;
    };
    const auto enter = [&] {  // the item's group and records
      const int g = active[in.item / blocks], nb = in.item % blocks;
      const int ex = a.map ? a.map[g] : g;
      in.row = max(0, a.offsets[g]);
      in.r1 = min(a.rows, a.offsets[g + 1]);
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
    // Tile `tile` of the cursor's step into slot `half` (of two); with tile
    // 0 the rows of x and the scales, into slot xs (of three).
    const auto copy_tile = [&](int half, int xs, int tile) {
      if (tile < left) {
        const uint32_t dst = codes + (half * kTiles + tile) * kTilePair;
        copy16(dst, p0 + tile * kTileBytes);
        copy16(dst + kTileBytes, p1 + tile * kTileBytes);
        if (tile == 0) {
          if (lane * 16 < kScaleRec) {
            const int at = min(left, kTiles) * kTileBytes;
            const uint32_t d =
                sc0 + xs * kWarps * 2 * kScaleRec + lane * 16;
            copy16(d, p0 + at);
            copy16(d + kScaleRec, p1 + at);
          }
          const int rows = min(a.x_rows, in.r1 - in.row) - x_first;
          const long long rest =  // of the rows from this lane's place on
              row_bytes - static_cast<long long>(in.step) * kStepBytes -
              lane * 16;
          const uint32_t d = x_dst + xs * m.x_slot;
#pragma unroll
          for (int r = 0; r < kRows; r += kRowStride)
            if (r < rows)
#pragma unroll
              for (int w = 0; w < kWords; w += 32)
                copy16_or_zero(d + r * kPitch + w * 16,
                               xp + r * row_bytes + w * 16, w * 16 < rest);
        }
      }
      copies_commit();
    };

    in.item = blockIdx.x;
    if (in.item < n_items && kw < n_steps) enter();
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int tile = 0; tile < kTiles; ++tile) copy_tile(s, s, tile);
      if (left > 0) advance();
    }

    // --- the computing side
    int half = 0, xs = 0;  // the slots of the step
    uint32_t x_row[NT];  // this lane's row of each eight
#pragma unroll
    for (int b = 0; b < NT; ++b)
      x_row[b] = sb + m.x + (kShareX ? 0 : warp * a.x_rows * kPitch) +
                 t * Rows<T>::kLaneBytes +
                 min(8 * b + c, a.x_rows - 1) * kPitch;
#pragma unroll 1
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
      const int g = active[item / blocks];
      const int r1 = min(a.rows, a.offsets[g + 1]);
#pragma unroll 1
      for (int row = max(0, a.offsets[g]); row < r1; row += a.x_rows) {
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
          Scales scale;
#pragma unroll
          for (int tile = 0; tile < kTiles; ++tile) {
            copies_wait<kRing - 1>();
            if (tile == 0) {
              if (kShareX)
                __syncthreads();
              else
                __syncwarp();
            }
            if (tile < tiles)
              multiply(one, acc, rows, w + tile * kTilePair, x_row, x0,
                       sc, tile, c, scale);
            // the slot's next tile: this lane has read what it overwrites
            copy_tile(half, next, tile);
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

  // Scales and zero operands of the group at hand, of both records.
  struct Scales {
    float s[2][2];
    uint32_t z[2][2];
  };

  // The groups that have rows and an expert, in order; their number.
  __device__ static int find_active(const GmmArgs& a, int32_t* active) {
    __shared__ int count[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int total = 0;
    for (int g0 = 0; g0 < a.n_groups; g0 += kThreads) {
      const int g = g0 + threadIdx.x;
      bool on = false;
      if (g < a.n_groups) {
        on = min(a.rows, a.offsets[g + 1]) > max(0, a.offsets[g]);
        const int ex = on && a.map ? a.map[g] : g < a.n_experts ? g : -1;
        if (on && (ex < 0 || ex >= a.n_experts)) {
          on = false;
          if (blockIdx.x == 0 && a.status)
            atomicOr(a.status, MOE_DEV_BAD_INDEX);
        }
      }
      const uint32_t vote = __ballot_sync(0xffffffffu, on);
      if (lane == 0) count[warp] = __popc(vote);
      __syncthreads();
      int before = total;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += count[w];
        total += count[w];
      }
      if (on) active[before + __popc(vote & ((1u << lane) - 1))] = g;
      __syncthreads();
    }
    return total;
  }

  // One tile of both records times the rows of x.
  __device__ static __forceinline__ void multiply(
      uint32_t one, float (&acc)[2][NT][4], int rows, uint32_t codes,
      const uint32_t (&x_row)[NT], uint32_t x0, uint32_t sc, int tile, int c,
      Scales& scale) {
    constexpr int GH = G == 32 ? 1 : 2;  // halves that share a scale
    const uint4 w[2] = {lds16(codes), lds16(codes + kTileBytes)};
#pragma unroll
    for (int h = 0; h < 2; h += GH) {
      const int g = (tile * kTileK + 32 * h) / G;
      uint32_t op[2][2 * GH][4], zero[2][4];
      float (&s)[2][2] = scale.s;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if ((tile * kTileK + 32 * h) % G == 0) {  // else the tile before's
          const uint32_t at = sc + r * kScaleRec;
          const uint32_t pair = lds4(at + g * 4);
          s[r][0] = __uint_as_float(pair << 16);
          s[r][1] = __uint_as_float(pair & 0xffff0000u);
          // -8 * (16 + zero); the stored byte is 8 * zero
          uint32_t z = 0x4040;
          if (Z) z = lds2(at + 32 * E + g * 2 - c * 2 * E);
          scale.z[r][0] = __byte_perm(z, 0xc3, 0x4040);
          scale.z[r][1] = __byte_perm(z, 0xc3, 0x4141);
        }
        zero[r][0] = zero[r][2] = scale.z[r][0];
        zero[r][1] = zero[r][3] = scale.z[r][1];
        const uint32_t words[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
        for (int i = 0; i < 2 * GH; ++i) expand(words[2 * h + i], one, op[r][i]);
      }
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        if (NT > 1 && 8 * b >= rows) break;
        float part[2][4] = {};
        Rows<T> v[GH];
        uint32_t o[Rows<T>::P][GH][4];
#pragma unroll
        for (int i = 0; i < GH; ++i) {
          v[i].load(x_row[b] + x0 + tile * kTileK * sizeof(T) +
                    (h + i) * 4 * Rows<T>::kLaneBytes);
#pragma unroll
          for (int p = 0; p < Rows<T>::P; ++p) v[i].part(p, o[p][i]);
        }
        // without zero points both records start from the same sums
#pragma unroll
        for (int r = 0; r < (Z ? 2 : 1); ++r)
#pragma unroll
          for (int i = 0; i < GH; ++i)
#pragma unroll
            for (int p = 0; p < Rows<T>::P; ++p) {
              mma(part[r], zero[r], o[p][i][0], o[p][i][1], part[r]);
              mma(part[r], zero[r], o[p][i][2], o[p][i][3], part[r]);
            }
#pragma unroll
        for (int r = 1; r >= 0; --r)
#pragma unroll
          for (int i = 0; i < GH; ++i)
#pragma unroll
            for (int p = 0; p < Rows<T>::P; ++p) {
              mma(part[r], op[r][2 * i], o[p][i][0], o[p][i][1],
                  part[!Z && r == 1 && i == 0 && p == 0 ? 0 : r]);
              mma(part[r], op[r][2 * i + 1], o[p][i][2], o[p][i][3], part[r]);
            }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[r][b][i] = fmaf(s[r][i >> 1], part[r][i], acc[r][b][i]);
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
              if (n < a.l.N) put(o + n, 0.125f * acc[h][b][i]);
            }
          }
        }
      return;
    }
    float* sums = reinterpret_cast<float*>(base + m.sums);
    constexpr int kRec = kRows * kTileN;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sums[(warp * 2 + h) * kRec +
               (8 * b + 2 * t + (i & 1)) * kTileN + c + 8 * (i >> 1)] =
              acc[h][b][i];
    __syncthreads();
    constexpr int kOut = NW * (DUAL ? 1 : 2) * kRec;
    for (int i = threadIdx.x; i < kOut; i += kThreads) {
      const int rec = i / kRec, r = i % kRec / kTileN, col = i % kTileN;
      const int w = DUAL ? rec : rec >> 1, h = DUAL ? 0 : rec & 1;
      const int n = n0 + rec * kTileN + col;
      if (r >= rows || n >= a.l.N) continue;
      float v = 0.0f, u = 0.0f;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const float* p = sums + ((k * NW + w) * 2 + h) * kRec + i % kRec;
        v += *p;
        if (DUAL) u += p[kRec];
      }
      put(out + static_cast<long long>(row + r) * a.l.N + n,
          DUAL ? swiglu(v, u) : 0.125f * v);
    }
    __syncthreads();
  }

  // of sums that are 8 times the products
  __device__ static __forceinline__ float swiglu(float g, float u) {
    g *= 0.125f;
    u *= 0.125f;
    return g / (1.0f + expf(-g)) * u;
  }
};

template <typename T, bool DUAL, int NW, int KW, int NT, int G, bool Z>
__global__ void __launch_bounds__(NW* KW * 32, NW* KW <= 8 ? 2 : 1)
    gmm_w4_kernel(const GmmArgs a) {
  Kernel<T, DUAL, NW, KW, NT, G, Z>::run(a);
}

struct Device {
  int sms = 0, smem = 0;
};
inline cudaError_t device(Device* d) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(
        &d->smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  return e;
}

template <typename T, bool DUAL, int NW, int KW, int NT, int G, bool Z>
cudaError_t launch_one(GmmArgs a, int tokens, const Device& d,
                       cudaStream_t s) {
  using Ker = Kernel<T, DUAL, NW, KW, NT, G, Z>;
  // routing gives a group at most one row of each token; float32 rows of
  // eight warps' k fill shared memory at half the rows
  a.x_rows = std::max(1, std::min(Ker::kRows, tokens));
  int bytes = Ker::smem(a.x_rows, a.n_groups).total;
  while (bytes + 1024 > d.smem && a.x_rows > 1) {
    a.x_rows /= 2;
    bytes = Ker::smem(a.x_rows, a.n_groups).total;
  }
  auto* kernel = gmm_w4_kernel<T, DUAL, NW, KW, NT, G, Z>;
  const cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const int per_sm =
      Ker::kThreads <= 256 && 2 * (bytes + 1024) <= d.smem ? 2 : 1;
  const long long items =
      static_cast<long long>((a.l.N + Ker::kCols - 1) / Ker::kCols) *
      std::min(a.n_groups, a.rows);
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>(items, static_cast<long long>(per_sm) * d.sms));
  kernel<<<grid, Ker::kThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool DUAL, int G, bool Z>
cudaError_t launch_shape(const GmmArgs& a, int tokens, cudaStream_t s) {
  Device d;
  const cudaError_t e = device(&d);
  if (e != cudaSuccess) return e;
  const long long groups = std::min(a.n_groups, a.rows);
  const long long items =
      groups * ((a.l.N + (DUAL ? 127 : 255)) / (DUAL ? 128 : 256));
  if (tokens <= 8 && items < 4ll * d.sms)
    return launch_one<T, DUAL, 1, 8, 1, G, Z>(a, tokens, d, s);
  if (sizeof(T) == 4 || a.rows <= 8 * groups)
    return launch_one<T, DUAL, 8, 1, 2, G, Z>(a, tokens, d, s);
  if constexpr (sizeof(T) == 2)
    return launch_one<T, DUAL, 16, 1, 4, G, Z>(a, tokens, d, s);
  return cudaErrorInvalidValue;
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
