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
//   idle lanes.  Codes become bf16 operands exactly: masked into the
//   mantissa of 128, they are 128 + code, and 128 + zero is subtracted.  The
//   scale multiplies the float32 partial sum of each 32 or 64 rows of W.
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
#include <cuda_bf16.h>

#include "w4.cuh"

namespace moe {
namespace {

using namespace w4;

constexpr int kTiles = kStepK / kTileK;  // tiles of a step
constexpr int kXSlots = 3;               // steps of x (and scales) in flight
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
// D += A B: A 16 weight columns x 16 k, B 16 k x 8 rows of x.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4],
                                    uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The operand registers of one word of codes: (code - zero) as bf16 pairs.
// zc and zd hold 128 + zero of columns c and c + 8, twice each.
__device__ __forceinline__ void expand(uint32_t w, uint32_t zc, uint32_t zd,
                                       uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t q = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const uint32_t z = i & 1 ? zd : zc;
    const __nv_bfloat162 v =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&q),
                *reinterpret_cast<const __nv_bfloat162*>(&z));
    a[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
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
  const char *p0, *p1;      // the warp's records (p1 may be null)
};

template <typename T, bool DUAL, int NW, int KW, int NT, int GH>
struct Kernel {
  static constexpr int kWarps = NW * KW;
  static constexpr int kThreads = kWarps * 32;
  static constexpr bool kShareX = NW > 1;  // else each warp copies its own k
  static constexpr int kRows = 8 * NT;
  static constexpr int kStepBytes = kStepK * sizeof(T);
  static constexpr int kPitch = kStepBytes + Rows<T>::kPad;
  // columns of an item
  static constexpr int kCols = DUAL ? NW * kTileN : 2 * NW * kTileN;
  static_assert(!kShareX || KW == 1, "x is shared by warps of the same k");

  // Shared memory: codes [warp][kRing][2][512], x [slot](or [slot][warp])
  // [rows][pitch], scales and zeros [slot][warp][2], sums, active groups.
  struct Smem {
    int x, x_slot, scales, scale_rec, scale_warp, sums, groups, total;
  };
  __host__ __device__ static Smem smem(const Layout& l, int x_rows,
                                       int n_groups) {
    Smem m;
    m.x = kWarps * kRing * 2 * kTileBytes;
    m.x_slot = (kShareX ? 1 : kWarps) * x_rows * kPitch;
    m.scales = m.x + kXSlots * m.x_slot;
    m.scale_rec = 8 * (kStepK / l.group) * (l.zeros ? 6 : 4);
    m.scale_warp = 2 * m.scale_rec;
    m.sums = m.scales + kXSlots * kWarps * m.scale_warp;
    m.groups = m.sums + (KW > 1 ? kWarps * 2 * kRows * kTileN * 4 : 0);
    m.total = m.groups + 4 * n_groups + 16;
    return m;
  }

  __device__ static void run(const GmmArgs& a) {
    extern __shared__ __align__(128) char base[];
    const Layout& l = a.l;
    const Smem m = smem(l, a.x_rows, a.n_groups);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nw = warp % NW, kw = warp / NW;
    const int c = lane >> 2, t = lane & 3;
    const int n_steps = (l.K + kStepK - 1) / kStepK, tiles_k = l.tiles_k();
    const uint32_t sb = smem_u32(base);
    int32_t* active = reinterpret_cast<int32_t*>(base + m.groups);
    const int n_active = find_active(a, active);

    const int blocks = (l.N + kCols - 1) / kCols;
    const int n_items = n_active * blocks;
    const uint32_t codes = sb + warp * (kRing * 2 * kTileBytes) + lane * 16;
    const int e = kStepK / l.group;  // groups of a step

    // --- the copies of one tile of a step (tile 0 brings x and the scales)
    Cursor in;
    const auto enter = [&](Cursor& q) {  // the item's group and records
      if (q.item >= n_items) return;
      const int g = active[q.item / blocks];
      const int nb = q.item % blocks;
      const int ex = a.map ? a.map[g] : g;
      q.row = max(0, a.offsets[g]);
      q.r1 = min(a.rows, a.offsets[g + 1]);
      const int rec = DUAL ? nb * NW + nw : 2 * (nb * NW + nw);
      const long long at = ex * l.matrix() + rec * l.record();
      q.p0 = rec < l.tiles_n() ? a.w0 + at : nullptr;
      if (DUAL)
        q.p1 = q.p0 ? a.w1 + at : nullptr;
      else
        q.p1 = rec + 1 < l.tiles_n() ? a.w0 + at + l.record() : nullptr;
    };
    const auto advance = [&](Cursor& q) {
      q.step += KW;
      if (q.step < n_steps) return;
      q.step = kw;
      q.row += a.x_rows;
      if (q.row < q.r1) return;
      q.item += gridDim.x;
      enter(q);
    };
    const auto copy_tile = [&](const Cursor& q, int slot, int tile) {
      if (q.item < n_items) {
        const int at = q.step * kTiles + tile;
        const uint32_t dst =
            codes + ((slot & 1) * kTiles + tile) * (2 * kTileBytes);
        if (at < tiles_k) {
          const long long src = static_cast<long long>(at) * kTileBytes +
                                lane * 16;
          if (q.p0) copy16(dst, q.p0 + src);
          if (q.p1) copy16(dst + kTileBytes, q.p1 + src);
        }
        if (tile == 0) {
          copy_x(a, q, sb + m.x + (slot % kXSlots) * m.x_slot, warp, lane);
          const uint32_t sc =
              sb + m.scales +
              ((slot % kXSlots) * kWarps + warp) * m.scale_warp;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const char* p = r == 0 ? q.p0 : q.p1;
            if (p) copy_scales(l, p, q.step, sc + r * m.scale_rec, c, t);
          }
        }
      }
      copies_commit();
    };

    in.item = blockIdx.x;
    in.step = kw;
    if (kw >= n_steps) in.item = n_items;  // no k for this warp
    enter(in);
    int in_slot = 0;
#pragma unroll 1
    for (; in_slot < 2; ++in_slot) {
#pragma unroll 1
      for (int tile = 0; tile < kTiles; ++tile) copy_tile(in, in_slot, tile);
      if (in.item < n_items) advance(in);
    }

    int slot = 0;
    Cursor q;
    q.item = blockIdx.x;
    q.step = kw;
    enter(q);
#pragma unroll 1
    while (q.item < n_items) {
      float acc[2][NT][4];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][b][i] = 0.0f;
      const int rows = min(a.x_rows, q.r1 - q.row);
#pragma unroll 1
      for (int step = kw; step < n_steps; step += KW, ++slot, ++in_slot) {
        const int xs = slot % kXSlots;
        const uint32_t xb =
            sb + m.x + xs * m.x_slot +
            (kShareX ? 0 : warp * a.x_rows * kPitch) + t * Rows<T>::kLaneBytes;
        const uint32_t sc = sb + m.scales +
                            (xs * kWarps + warp) * m.scale_warp;
#pragma unroll 1
        for (int tile = 0; tile < kTiles; ++tile) {
          copies_wait<kRing - 1>();
          if (tile == 0) {
            if (kShareX)
              __syncthreads();
            else
              __syncwarp();
          }
          if (step * kTiles + tile < tiles_k)
            multiply(a, m, acc, rows,
                     codes + ((slot & 1) * kTiles + tile) * (2 * kTileBytes),
                     xb + tile * (kTileK * static_cast<int>(sizeof(T))), sc,
                     tile, c, e);
          // the slot's next tile: this lane has read what it overwrites
          copy_tile(in, in_slot, tile);
        }
        if (in.item < n_items) advance(in);
      }
      finish(a, m, acc, q, blocks, rows, base, warp, nw, kw, c, t);
      // next rows of the group, or the next item
      q.row += a.x_rows;
      if (q.row >= q.r1) {
        q.item += gridDim.x;
        enter(q);
      }
    }
    copies_wait<0>();
  }

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

  __device__ static __forceinline__ void copy_x(const GmmArgs& a,
                                                const Cursor& q, uint32_t dst,
                                                int warp, int lane) {
    constexpr int kWords = kStepBytes / 16;  // of a row
    const int rows = min(a.x_rows, q.r1 - q.row);
    const int first = kShareX ? threadIdx.x : lane;
    constexpr int kStride = kShareX ? kThreads : 32;
    if (!kShareX) dst += warp * a.x_rows * kPitch;
    const long long pitch = static_cast<long long>(a.l.K) * sizeof(T);
    for (int i = first; i < rows * kWords; i += kStride) {
      const int r = i / kWords, w = i % kWords;
      const long long at = static_cast<long long>(q.step) * kStepBytes +
                           w * 16;
      const bool in = at < pitch;
      copy16_or_zero(dst + r * kPitch + w * 16,
                     a.x + (q.row + r) * pitch + (in ? at : 0), in);
    }
  }

  // The scales (zeros) of a step: e pairs of bf16 (bytes) for each c.
  __device__ static __forceinline__ void copy_scales(const Layout& l,
                                                     const char* rec,
                                                     int step, uint32_t dst,
                                                     int c, int t) {
    const int e = kStepK / l.group, at = c * l.stored_groups() + step * e;
    const char* s = rec + l.scales_at() + 4ll * at;
    const char* z = rec + l.zeros_at() + 2ll * at;
    const uint32_t ds = dst + c * 4 * e, dz = dst + 32 * e + c * 2 * e;
    if (e == 8) {
      if (t < 2) copy16(ds + 16 * t, s + 16 * t);
      if (t == 2 && l.zeros) copy16(dz, z);
    } else if (e == 4) {
      if (t == 0) copy16(ds, s);
      if (t == 2 && l.zeros) copy8(dz, z);
    } else {
      if (t == 0) copy8(ds, s);
      if (t == 2 && l.zeros) copy4(dz, z);
    }
  }

  // One tile of both records times the rows of x.
  __device__ static __forceinline__ void multiply(
      const GmmArgs& a, const Smem& m, float (&acc)[2][NT][4], int rows,
      uint32_t codes, uint32_t x, uint32_t sc, int tile, int c, int e) {
    const uint4 w[2] = {lds16(codes), lds16(codes + kTileBytes)};
#pragma unroll
    for (int h = 0; h < 2; h += GH) {  // GH halves share a scale
      uint32_t op[2][2 * GH][4];
      float s[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int g = (tile * kTileK + 32 * h) / a.l.group;
        const uint32_t pair = lds4(sc + r * m.scale_rec + (c * e + g) * 4);
        s[r][0] = __uint_as_float(pair << 16);
        s[r][1] = __uint_as_float(pair & 0xffff0000u);
        uint32_t zc = 0x43084308u, zd = 0x43084308u;  // 136: zero 8
        if (a.l.zeros) {
          const uint32_t z =
              lds2(sc + r * m.scale_rec + 32 * e + (c * e + g) * 2);
          zc = __byte_perm(z, 0x43, 0x4040);
          zd = __byte_perm(z, 0x43, 0x4141);
        }
        const uint32_t words[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
        for (int i = 0; i < 2 * GH; ++i) expand(words[2 * h + i], zc, zd, op[r][i]);
      }
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        if (NT > 1 && 8 * b >= rows) break;
        const uint32_t xr = x + min(8 * b + c, a.x_rows - 1) * kPitch;
        float part[2][4] = {};
#pragma unroll
        for (int i = 0; i < GH; ++i) {
          Rows<T> v;
          v.load(xr + (h + i) * 4 * Rows<T>::kLaneBytes);
#pragma unroll
          for (int p = 0; p < Rows<T>::P; ++p) {
            uint32_t o[4];
            v.part(p, o);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              mma(part[r], op[r][2 * i], o[0], o[1]);
              mma(part[r], op[r][2 * i + 1], o[2], o[3]);
            }
          }
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
      const GmmArgs& a, const Smem& m, const float (&acc)[2][NT][4],
      const Cursor& q, int blocks, int rows, char* base, int warp, int nw,
      int kw, int c, int t) {
    T* out = static_cast<T*>(a.out);
    const int n0 = (q.item % blocks) * kCols;
    if (KW == 1) {
      // a lane holds rows 2t and 2t + 1 of each 8, columns c and c + 8
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * b + 2 * t + (i & 1);
          if (r >= rows) continue;
          const int col = c + 8 * (i >> 1);
          T* o = out + static_cast<long long>(q.row + r) * a.l.N;
          if (DUAL) {
            const int n = n0 + nw * kTileN + col;
            if (n < a.l.N) put(o + n, swiglu(acc[0][b][i], acc[1][b][i]));
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int n = n0 + (2 * nw + h) * kTileN + col;
              if (n < a.l.N) put(o + n, acc[h][b][i]);
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
      put(out + static_cast<long long>(q.row + r) * a.l.N + n,
          DUAL ? swiglu(v, u) : v);
    }
    __syncthreads();
  }

  __device__ static __forceinline__ float swiglu(float g, float u) {
    return g / (1.0f + expf(-g)) * u;
  }
};

template <typename T, bool DUAL, int NW, int KW, int NT, int GH>
__global__ void __launch_bounds__(NW* KW * 32, NW* KW <= 8 ? 2 : 1)
    gmm_w4_kernel(const GmmArgs a) {
  Kernel<T, DUAL, NW, KW, NT, GH>::run(a);
}

struct Device {
  int sms = 0, smem = 0;
};
cudaError_t device(Device* d) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(
        &d->smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  return e;
}

template <typename T, bool DUAL, int NW, int KW, int NT, int GH>
cudaError_t launch_one(GmmArgs a, int tokens, cudaStream_t s) {
  using Ker = Kernel<T, DUAL, NW, KW, NT, GH>;
  Device d;
  cudaError_t e = device(&d);
  if (e != cudaSuccess) return e;
  // routing gives a group at most one row of each token; float32 rows of
  // eight warps' k fill shared memory at half the rows
  a.x_rows = std::max(1, std::min(Ker::kRows, tokens));
  int bytes = Ker::smem(a.l, a.x_rows, a.n_groups).total;
  while (bytes + 1024 > d.smem && a.x_rows > 1) {
    a.x_rows /= 2;
    bytes = Ker::smem(a.l, a.x_rows, a.n_groups).total;
  }
  auto* kernel = gmm_w4_kernel<T, DUAL, NW, KW, NT, GH>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           bytes);
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

template <typename T, bool DUAL, int GH>
cudaError_t launch_shape(const GmmArgs& a, int tokens, cudaStream_t s) {
  Device d;
  const cudaError_t e = device(&d);
  if (e != cudaSuccess) return e;
  const long long groups = std::min(a.n_groups, a.rows);
  const long long items =
      groups * ((a.l.N + (DUAL ? 127 : 255)) / (DUAL ? 128 : 256));
  if (tokens <= 8 && items < 4ll * d.sms)
    return launch_one<T, DUAL, 1, 8, 1, GH>(a, tokens, s);
  if (sizeof(T) == 4 || a.rows <= 8 * groups)
    return launch_one<T, DUAL, 8, 1, 2, GH>(a, tokens, s);
  if constexpr (sizeof(T) == 2)
    return launch_one<T, DUAL, 16, 1, 4, GH>(a, tokens, s);
  return cudaErrorInvalidValue;
}

template <bool DUAL>
cudaError_t launch(const moe_config_t& c, const GmmArgs& a, cudaStream_t s) {
  const bool fine = a.l.group == 32;
  if (c.dtype == MOE_F32)
    return fine ? launch_shape<float, DUAL, 1>(a, c.T, s)
                : launch_shape<float, DUAL, 2>(a, c.T, s);
  return fine ? launch_shape<__nv_bfloat16, DUAL, 1>(a, c.T, s)
              : launch_shape<__nv_bfloat16, DUAL, 2>(a, c.T, s);
}

GmmArgs args_of(const moe_config_t& c, const moe_w4_t& o, const Groups& g,
                const int32_t* offsets, int K, int N, int32_t* status) {
  GmmArgs a = {};
  a.offsets = offsets;
  a.map = g.map;
  a.status = status;
  a.l = layout(o, K, N);
  a.n_experts = c.E;
  a.n_groups = g.n;
  a.rows = c.T * c.k;
  return a;
}

moe_status_t gate_up(const moe_config_t& c, const moe_w4_t& o,
                     const Groups& g, const void* x, const int32_t* offsets,
                     const void* wg, const void* wu, void* h, int32_t* status,
                     cudaStream_t s) {
  GmmArgs a = args_of(c, o, g, offsets, c.H, c.F, status);
  a.x = static_cast<const char*>(x);
  a.w0 = static_cast<const char*>(wg);
  a.w1 = static_cast<const char*>(wu);
  a.out = h;
  return launch<true>(c, a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t down(const moe_config_t& c, const moe_w4_t& o, const Groups& g,
                  const void* h, const int32_t* offsets, const void* wd,
                  void* y, int32_t* status, cudaStream_t s) {
  GmmArgs a = args_of(c, o, g, offsets, c.F, c.H, status);
  a.x = static_cast<const char*>(h);
  a.w0 = static_cast<const char*>(wd);
  a.out = y;
  return launch<false>(c, a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t check(const moe_config_t* cfg, const moe_w4_t* opt,
                   int32_t n_groups, const int32_t* map, Groups* g) {
  const moe_status_t st = validate(cfg);
  if (st != MOE_OK) return st;
  if (!w4::options_ok(opt) || cfg->F < 1 ||
      !groups_of(*cfg, n_groups, map, g))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_gmm_gate_up_w4(const moe_config_t* cfg, const moe_w4_t* opt,
                                int32_t n_groups, const int32_t* group_expert,
                                const void* x_sorted,
                                const int32_t* group_offsets,
                                const void* w_gate, const void* w_up, void* h,
                                int32_t* status_word, moe_stream_t stream) {
  Groups g;
  const moe_status_t st = check(cfg, opt, n_groups, group_expert, &g);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ok_ptr(x_sorted, true) || !ok_ptr(group_offsets, false) ||
      !ok_ptr(w_gate, true) || !ok_ptr(w_up, true) || !ok_ptr(h, true))
    return MOE_ERR_INVALID_ARG;
  return gate_up(*cfg, *opt, g, x_sorted, group_offsets, w_gate, w_up, h,
                 status_word, stream);
}

moe_status_t moe_gmm_down_w4(const moe_config_t* cfg, const moe_w4_t* opt,
                             int32_t n_groups, const int32_t* group_expert,
                             const void* h, const int32_t* group_offsets,
                             const void* w_down, void* y_sorted,
                             int32_t* status_word, moe_stream_t stream) {
  Groups g;
  const moe_status_t st = check(cfg, opt, n_groups, group_expert, &g);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ok_ptr(h, true) || !ok_ptr(group_offsets, false) ||
      !ok_ptr(w_down, true) || !ok_ptr(y_sorted, true))
    return MOE_ERR_INVALID_ARG;
  return down(*cfg, *opt, g, h, group_offsets, w_down, y_sorted, status_word,
              stream);
}

moe_status_t moe_gmm_swiglu_w4(const moe_config_t* cfg, const moe_w4_t* opt,
                               const void* x_sorted,
                               const int32_t* group_offsets,
                               const void* w_gate, const void* w_up,
                               const void* w_down, void* h, void* y_sorted,
                               int32_t* status_word, moe_stream_t stream) {
  Groups g;
  const moe_status_t st = check(cfg, opt, 0, nullptr, &g);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ok_ptr(x_sorted, true) || !ok_ptr(group_offsets, false) ||
      !ok_ptr(w_gate, true) || !ok_ptr(w_up, true) ||
      !ok_ptr(w_down, true) || !ok_ptr(h, true) || !ok_ptr(y_sorted, true))
    return MOE_ERR_INVALID_ARG;
  const moe_status_t up = gate_up(*cfg, *opt, g, x_sorted, group_offsets,
                                  w_gate, w_up, h, status_word, stream);
  if (up != MOE_OK) return up;
  return down(*cfg, *opt, g, h, group_offsets, w_down, y_sorted, status_word,
              stream);
}

}  // extern "C"
