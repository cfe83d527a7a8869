// Products of the routed rows with microscaled 4-bit experts on tcgen05, rows
// and weights both in 4 bits (mx.cuh has the formats and the layout).
//
//   gate_up: h[r] = silu(x[r] Wg) * (x[r] Wu), quantised again
//   down:    y[r] = h[r] Wd
//
// The block-scaled matrix instruction multiplies 64 of k of both operands and
// their scales at once, so nothing is expanded.  128 columns of weights are
// its M rows and the rows of x its N columns: a group of few rows costs few
// columns, and one of any number of rows splits at any multiple of 16.
//
// A CTA an SM walks over items, a tile of 128 columns (of the gate and the up
// matrix, or of the down matrix) for up to NT = 64 rows of one group:
//   * a thread brings the weights' records by bulk copy and the rows' codes by
//     TMA, 256 of k a stage (rows past the group's are other groups' or zeros;
//     they reach only columns that are not written);
//   * four warps (or eight in turn), one for each quarter of the lanes of tensor
//     memory, write a stage's scales there, those of the weights from shared memory and those
//     of the rows from global memory;
//   * a warp issues the matrix instructions;
//   * four warps, or eight or sixteen, turn the sums into rows of the output, a
//     thread a column, while the next item's sums go to the other accumulator,
//     if there is one.
// Every wait is bounded; one that gives up raises MOE_DEV_TIMEOUT and the CTA
// drains and returns.
//
// With many rows a group, what a CTA brings and reads for a matrix instruction
// bounds it, so two SMs work on one item as a pair: up to 192 rows by 256 columns
// of weights, half of the columns in each CTA, and the rows' codes halved
// between them, which the instruction reads from both.  One CTA's warp issues
// for both.
//
// Measured, quantising the rows and both products: one token, 8 experts of 7168
// x 2048, blocks of 16, 198 MB, 42 us (4.7 TB/s; 128 items leave 24 of 152 SMs
// idle in the first product); 64 tokens over 146 such experts, blocks of 32, 546
// to 589 us (5.6 to 6.1 TB/s, with where the buffers lie); 16 experts of 5120 x
// 8192, a row each, 149 to 173.  32768 rows over 32 experts of 7168 x 2048, blocks
// of 16, 884 to 891 us: quantising the rows 128, gate and up 438 to 441 (4.4
// PFLOP/s), down 338 (2.8 PFLOP/s).  At a step before, of 444 and 338, 385 and 297
// were left if nothing read the sums, 369 and 266 without matrix instructions,
// 235 and 217 if scales were not loaded either.
#pragma once

#include <atomic>

#include "chunks.cuh"
#include "launch.cuh"
#include "mx.cuh"
#include "tc_common.cuh"

namespace moe {
namespace tc {
// The GEMMs' test hook (gmm_tc.cu): stop the producer after this many stage
// fills (-1: never), so that the next wait runs out.
extern std::atomic<long long> g_stall_after_fills;
}  // namespace tc

namespace mx {

using launch::Device;

struct GmmArgs {
  const int32_t *offsets, *map;
  const uint8_t* x_scales;
  const char *w0, *w1;
  const float *s0, *s1;  // the matrices' scales [E], or null
  float x_scale;
  float inv_out;         // gate_up: 1 / h_scale
  uint8_t *h_codes, *h_scales;
  void* y;
  int32_t* status;
  Layout l;
  int n_experts, n_groups, rows, chunk, chunks;
  int tokens;  // routing gives a group at most one row of each
  bool f32;    // y's type
  bool early;  // may read all but the rows before the kernel that writes those
               // has ended
  long long stall_after_fills;  // tests of the timeout path only (-1: off)
};

// The launch of either product (gmm_mx_*.cu).
cudaError_t launch_gmm_mx_gate_up(const GmmArgs& a, const void* codes,
                                  cudaStream_t s);
cudaError_t launch_gmm_mx_down(const GmmArgs& a, const void* codes,
                               cudaStream_t s);

// Whether passes of 192 rows on SM pairs are faster than passes of 64 on single
// SMs: by the mean rows of a group, where groups can have more than 64 (routing
// gives a group at most one row of each token).  32 experts of 7168 x 2048, rows
// quantised and both products, singles against pairs: 32 rows a group 169 and 171
// us, 48 rows 173 and 177, 64 rows 194 and 181, 128 rows 300 and 198, 1024 rows
// 1872 and 890.  (Passes of 16 rows gained nothing: 113 us for one row a group, 114
// in passes of 64.)  Those groups are alike.  The mean counts empty groups and does
// not see a popular one: 256 experts, blocks of 32, 1024 tokens x 8 (a mean of 32)
// take 1015 us if drawn alike and 1154 by Zipf's law, where one expert has 810
// rows in passes of 64; 4096 tokens 1175 and 1435.
inline bool many_rows(const GmmArgs& a) {
  return a.tokens > 64 &&
         a.rows > 48ll * std::min(a.n_groups, a.rows);
}

constexpr int kScaleWarps = 4;
constexpr int kMaxSplits = 512;
constexpr int kMaxChunks = kMaxExperts + kMaxSplits;
constexpr int kMaxShared = 226 * 1024;
constexpr int kMaxStages = 8;
constexpr int kBarBytes = 256;

// ---------------------------------------------------------------- PTX ----
// Bytes from global to shared memory, in one piece (16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src,
                                          uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// Columns of this warp's quarter of the lanes, 8 or 16 at a time.
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&r)[N]) {
  static_assert(N == 8 || N % 16 == 0, "columns of scales");
  if constexpr (N == 8) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, "
        "%6, %7, %8};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
        "r"(r[6]), "r"(r[7])
        : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 16)
      asm volatile(
          "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, "
          "%6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at + i),
          "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]),
          "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7]),
          "r"(r[i + 8]), "r"(r[i + 9]), "r"(r[i + 10]), "r"(r[i + 11]),
          "r"(r[i + 12]), "r"(r[i + 13]), "r"(r[i + 14]), "r"(r[i + 15])
          : "memory");
  }
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
// A bounded wait as tc::mbar_wait, but the clock is read only after many looks
// in vain: reading it takes longer than most of these waits.
static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag,
                                              int32_t* status) {
  uint64_t t0 = 0;
  for (uint32_t looks = 1;; ++looks) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((looks & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t t = tc::globaltimer();
      if (t0 == 0) t0 = t;
      if (t - t0 > tc::kWaitLimitNs) {
        *abort_flag = 1;
        if (status) atomicOr(status, MOE_DEV_TIMEOUT);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity,
                                     volatile int* abort_flag,
                                     int32_t* status) {
  return tc::mbar_try_wait(bar, parity) ||
         wait_long(bar, parity, abort_flag, status);
}

// D (+)= A B over 64 of k, both 4-bit in shared memory, each block of BLOCK of
// k times its scales in tensor memory; of a pair of CTAs, A's rows and D's in
// halves, B's columns too, and the scales of B whole in both.
template <int BLOCK>
__device__ __forceinline__ void umma_mx_pair(uint32_t d, uint64_t a,
                                             uint64_t b, uint32_t idesc,
                                             uint32_t sa, uint32_t sb,
                                             uint32_t accumulate) {
  if (BLOCK == 16)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
template <int BLOCK>
__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t a, uint64_t b,
                                        uint32_t idesc, uint32_t sa,
                                        uint32_t sb, uint32_t accumulate) {
  if (BLOCK == 16)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// Instruction descriptor of the block-scaled kinds: B's scale word's first
// byte (bits 4-5), A and B of the 4-bit type (1 in bits 7-9 and 10-12), N >> 3
// in bits 17-22, scales a power of two (bit 23), M >> 7 in bits 27-28, A's
// scale word's first byte (bits 29-30).
__device__ __forceinline__ uint32_t idesc_mx(int block, int m, int n) {
  return 1u << 7 | 1u << 10 | static_cast<uint32_t>(n >> 3) << 17 |
         (block == 32 ? 1u << 23 : 0u) | static_cast<uint32_t>(m >> 7) << 27;
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, "
      "%7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(at)
      : "memory");
}
// The registers of the loads before it are there.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
                 "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// ------------------------------------------------------------- kernel ----
template <bool DUAL, int BLOCK, int NT, bool PAIR>
struct Gmm {
  static constexpr int kCtas = PAIR ? 2 : 1;  // of an item
  // Warps for each quarter of the lanes, which share an item's rows.  Many rows
  // of both matrices leave tensor memory no second accumulator, and the matrix
  // instructions wait while it is read: 10.8 us of an item's 29 with one warp
  // a quarter, 7 of 25 with four (32768 rows; a run that read no sums
  // subtracted), 2.5 of 21 as it is now.  Down has a second one: 397, 391, 422,
  // 453 us with one to four, at that step.
  static constexpr int kRowParts = !PAIR ? 1 : DUAL ? 4 : 2;
  static constexpr int kEpiWarps = 4 * kRowParts;
  static constexpr int kLoadWarp = kEpiWarps;
  static constexpr int kMmaWarp = kLoadWarp + 1;
  static constexpr int kScaleWarp = kMmaWarp + 1;
  // Four warps write scales to tensor memory; where rows are many, whose stages
  // are short, two such teams do so in turn, each every other stage (down, 32768
  // rows: 391 us with one, 360 with two, 338 with the rows' scales written before
  // the stage is there, 346 with four).  Gate and up have no registers for two:
  // 455 us against 438 (with one, 80 registers and 44 bytes spilled in blocks of
  // 16, 20 in blocks of 32).
  static constexpr int kTeams = PAIR && !DUAL ? 2 : 1;
  static constexpr int kWarps = kScaleWarp + kScaleWarps * kTeams;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kMats = DUAL ? 2 : 1;
  static constexpr int kTiles = scale_tiles(BLOCK);  // of 128 rows, a stage
  static constexpr int kRec = record_bytes(BLOCK);
  // Tiles of the rows' scales, as the weights'.  (32 rows would fit the four
  // columns of one tile, a column for each 64 of k; but the instruction wants
  // its scales at a multiple of four columns.)
  static constexpr int kRowTiles = (NT + 127) / 128 * kTiles;
  // Rows of one TMA copy: few where rows are few; where they are many, small
  // copies are what takes the time.
  static constexpr int kRowBox = PAIR ? NT / 4 : 16;
  static constexpr int kX = kMats * kRec;  // the rows' codes
  static constexpr int kStage = kX + NT / kCtas * 128;
  static constexpr int kRoom = kMaxShared - 1024 - kBarBytes - 8 * kMaxChunks;
  static constexpr int kStages =
      kRoom / kStage < kMaxStages ? kRoom / kStage : kMaxStages;
  static_assert(kStages >= 3, "copies stay ahead");
  static_assert(kRec % 1024 == 0 && NT % (16 * kCtas) == 0 &&
                    kRowBox % 8 == 0 && NT / kCtas % kRowBox == 0,
                "swizzled tiles aligned");
  // Tensor memory: accumulators [buffer][matrix][NT], then scales [buffer]
  // of the weights [matrix][tile][4] and the rows [tile][4], both from a
  // multiple of 16 columns.
  static constexpr int kAcc = kMats * NT;
  static constexpr int kScaleA = 4 * kTiles;
  static constexpr int kScaleX = (kMats * kScaleA + 15) / 16 * 16;
  static constexpr int kScales = kScaleX + (4 * kRowTiles + 15) / 16 * 16;
  static constexpr int kBuffers = 2 * kAcc + 2 * kScales <= 512 ? 2 : 1;
  static constexpr int kScaleAt = kBuffers * kAcc;
  static constexpr int kFit = (512 - kScaleAt) / kScales;
  static constexpr int kScaleBufs = kFit < kStages ? kFit : kStages;
  static_assert(kScaleBufs >= 2, "tensor memory");

  static constexpr int shared_bytes(int chunks) {
    return 1024 + kStages * kStage + kBarBytes + 8 * chunks;
  }

  // Scales have barriers of their own, one for each of their buffers.
  struct Bars {
    uint32_t full, scales, empty, acc_full, acc_empty, done;
  };
  // Where a role stands in a ring of N buffers.
  template <int N = kStages>
  struct Ring {
    int st = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
      if (++st == N) {
        st = 0;
        phase ^= 1;
      }
    }
  };
  struct Item {
    int tile, expert, row, rows;
  };
  __device__ static __forceinline__ Item item_at(const GmmArgs& a,
                                                 const int2* chunks, int i,
                                                 int tiles) {
    const int2 c = chunks[i / tiles];
    return {i % tiles * kCtas + rank(), a.map ? a.map[c.x] : c.x, c.y,
            chunk_end(a, c) - c.y};
  }
  // This CTA of its pair.
  __device__ static __forceinline__ int rank() {
    return PAIR ? blockIdx.x & 1 : 0;
  }
  // Columns of the instruction for so many rows.
  __device__ static __forceinline__ int columns(int rows) {
    return (rows + 16 * kCtas - 1) / (16 * kCtas) * (16 * kCtas);
  }
  // Calls f(item) for the passes of up to NT rows of this CTA's items until
  // it returns false.
  template <typename F>
  __device__ static __forceinline__ void passes(const GmmArgs& a,
                                                const int2* chunks,
                                                int n_items, int tiles,
                                                const F& f) {
#pragma unroll 1
    for (int i = blockIdx.x / kCtas; i < n_items; i += gridDim.x / kCtas) {
      Item it = item_at(a, chunks, i, tiles);
      const int end = it.row + it.rows;
#pragma unroll 1
      for (; it.row < end; it.row += NT) {
        it.rows = min(NT, end - it.row);
        if (!f(it)) return;
      }
    }
  }
  __device__ static __forceinline__ bool wait_all(uint32_t bar, uint32_t phase,
                                                  volatile int* abort_flag,
                                                  int32_t* status) {
    return __all_sync(0xffffffffu, wait(bar, phase, abort_flag, status));
  }

  __device__ static void run(const GmmArgs& a, const CUtensorMap* map) {
    extern __shared__ __align__(1024) char raw[];
    char* base = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
    __shared__ int abort_word;
    __shared__ uint32_t tmem_word;
    volatile int* abort_flag = &abort_word;
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const uint32_t sb = tc::smem_u32(base);
    Bars b;
    b.full = sb + kStages * kStage;
    b.scales = b.full + 8 * kStages;
    b.empty = b.scales + 8 * kScaleBufs;
    b.acc_full = b.empty + 8 * kStages;
    b.acc_empty = b.acc_full + 8 * kBuffers;
    b.done = b.acc_empty + 8 * kBuffers;
    if (threadIdx.x == 0) {
      abort_word = 0;
      for (int i = 0; i < kStages; ++i) {
        tc::mbar_init(b.full + 8 * i, 1);
        tc::mbar_init(b.empty + 8 * i, 1);
      }
      // (the first CTA's count both CTAs' warps)
      for (int i = 0; i < kScaleBufs; ++i)
        tc::mbar_init(b.scales + 8 * i, kScaleWarps * kCtas);
      for (int i = 0; i < kBuffers; ++i) {
        tc::mbar_init(b.acc_full + 8 * i, 1);
        tc::mbar_init(b.acc_empty + 8 * i, kEpiWarps * kCtas);
      }
      tc::mbar_init(b.done, 1);
      tc::fence_barrier_init();
      tc::fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
      if (PAIR) {
        tc::tmem_alloc_pair(tc::smem_u32(&tmem_word), tc::kTmemCols);
        tc::tmem_relinquish_pair();
      } else {
        tc::tmem_alloc(tc::smem_u32(&tmem_word), tc::kTmemCols);
        tc::tmem_relinquish();
      }
    }
    // Offsets and weights were final before the kernel that writes the rows
    // began, where this one may start early; else nothing is read before all
    // kernels before it have ended.
    if (!a.early) launch::wait_for_previous();
    int2* chunks =
        reinterpret_cast<int2*>(base + kStages * kStage + kBarBytes);
    const int n_chunks = find_chunks<kWarps>(a, chunks);  // barriers within
    tc::tc_fence_before();
    __syncthreads();
    if (PAIR) tc::cluster_sync();  // both CTAs' barriers exist
    tc::tc_fence_after();
    launch::let_next_start();
    const uint32_t tmem = tmem_word;
    const int tiles = (a.l.tiles_n() + kCtas - 1) / kCtas;
    const int n_items = n_chunks * tiles;
    if (warp < kEpiWarps)
      write_out(a, b, chunks, n_items, tiles, tmem, warp, lane, abort_flag);
    else if (warp == kLoadWarp)
      load(a, map, sb, b, chunks, n_items, tiles, lane, abort_flag);
    else if (warp == kMmaWarp)
      multiply(a, sb, b, chunks, n_items, tiles, tmem, lane, abort_flag);
    else
      load_scales(a, sb, b, chunks, n_items, tiles, tmem, warp & 3,
                  (warp - kScaleWarp) / kScaleWarps, lane, abort_flag);
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    // neither CTA leaves while the other may still use what is its
    if (PAIR) tc::cluster_sync();
    tc::tc_fence_after();
    if (warp == kMmaWarp) {
      if (PAIR)
        tc::tmem_dealloc_pair(tmem, tc::kTmemCols);
      else
        tc::tmem_dealloc(tmem, tc::kTmemCols);
    }
  }

  // ---- weights and the rows' codes
  __device__ static void load(const GmmArgs& a, const CUtensorMap* map,
                              uint32_t sb, const Bars& b, const int2* chunks,
                              int n_items, int tiles, int lane,
                              volatile int* abort_flag) {
    if (lane != 0) return;
    const int stages = a.l.stages();
    Ring<> ring;
    ring.phase = 1;
    long long filled = 0;
    const auto weights = [&](const Item& it, int s, int st) {
      // (the second of a pair may be past the last tile: it has the last
      // again, and writes nothing)
      const int tile = PAIR ? min(it.tile, a.l.tiles_n() - 1) : it.tile;
      const long long at = it.expert * a.l.matrix() + tile * a.l.tile() +
                           static_cast<long long>(s) * kRec;
      const uint32_t dst = sb + st * kStage, bar = b.full + 8 * st;
      const int boxes =
          (columns(it.rows) / kCtas + kRowBox - 1) / kRowBox;
      tc::mbar_expect_tx(bar, kMats * kRec + boxes * kRowBox * 128);
      bulk_load(dst, a.w0 + at, kRec, bar);
      if (DUAL) bulk_load(dst + kRec, a.w1 + at, kRec, bar);
    };
    const auto rows = [&](const Item& it, int s, int st) {
      const uint32_t dst = sb + st * kStage + kX, bar = b.full + 8 * st;
      const int n = columns(it.rows) / kCtas;
#pragma unroll 1
      for (int r = 0; r < n; r += kRowBox)
        tc::tma_load_2d(dst + r * 128, map, bar, s * (kStageK / 2),
                        it.row + rank() * n + r);
    };
    // The weights of the first stages do not wait for the kernel that writes
    // the rows.
    int ahead = 0;
    if (a.stall_after_fills < 0)
      passes(a, chunks, n_items, tiles, [&](const Item& it) {
        for (int s = 0; s < stages && ahead < kStages; ++s, ++ahead)
          weights(it, s, ahead);
        return ahead < kStages;
      });
    launch::wait_for_previous();
    passes(a, chunks, n_items, tiles, [&](const Item& it) {
#pragma unroll 1
      for (int s = 0; s < stages; ++s) {
        if (a.stall_after_fills >= 0 && filled >= a.stall_after_fills)
          return false;
        if (filled >= ahead) {
          if (!wait(b.empty + 8 * ring.st, ring.phase, abort_flag, a.status))
            return false;
          weights(it, s, ring.st);
        }
        rows(it, s, ring.st);
        ++filled;
        ring.next();
      }
      return true;
    });
    // This thread's last copies must have landed before the CTA ends.  The
    // instructions that read them wait for them, unless a wait of any warp
    // gave up: also after this thread's last fill.
    for (long long i = 0; i < filled && i < kStages; ++i) {
      if (--ring.st < 0) {
        ring.st = kStages - 1;
        ring.phase ^= 1;
      }
      tc::mbar_wait(b.full + 8 * ring.st, ring.phase ^ 1, nullptr, a.status);
    }
  }

  // ---- scales to tensor memory.  The instruction reads them from every
  // quarter of the lanes, so each of the four warps writes all of them to its
  // own quarter.  (The tensor cores can copy them from shared memory to all
  // quarters, but a copy of 512 bytes takes its turn among the matrix
  // instructions: 45 clocks, beside 60 to 90 for one of those.)
  __device__ static void load_scales(const GmmArgs& a, uint32_t sb,
                                     const Bars& b, const int2* chunks,
                                     int n_items, int tiles, uint32_t tmem,
                                     int quarter, int team, int lane,
                                     volatile int* abort_flag) {
    constexpr int kRows = (NT + 31) / 32;  // rows a lane
    const int stages = a.l.stages(), groups = a.l.K / BLOCK;
    const uint32_t out =
        tmem + kScaleAt + (static_cast<uint32_t>(32 * quarter) << 16);
    Ring<> ring, back;
    Ring<kScaleBufs> sring;
    int lead = 0;  // stages so far, counted up to kScaleBufs
    // The words of rows lane, lane + 32, .. of a stage; zeros past the rows.
    const auto load = [&](const Item& it, int s, uint32_t (&v)[kRows][kTiles]) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = i * 32 + lane;
        const uint8_t* p =
            a.x_scales + (static_cast<long long>(s) * a.rows + it.row + r) *
                             (4 * kTiles);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) v[i][j] = 0;
        if (r >= it.rows) continue;
        if constexpr (kTiles == 4) {
          const uint4 w = *reinterpret_cast<const uint4*>(p);
          v[i][0] = w.x, v[i][1] = w.y, v[i][2] = w.z, v[i][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(p);
          v[i][0] = w.x, v[i][1] = w.y;
        }
      }
      // what lies behind a row's last scale counts as zero
      if (s == stages - 1 && groups % (4 * kTiles) != 0) {
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          const int left = groups - (s * kTiles + j) * 4;
          if (left < 4) {
            const uint32_t mask = left > 0 ? (1u << (8 * left)) - 1 : 0u;
#pragma unroll
            for (int i = 0; i < kRows; ++i) v[i][j] &= mask;
          }
        }
      }
    };
    launch::wait_for_previous();
    passes(a, chunks, n_items, tiles, [&](const Item& it) {
      uint32_t next[kRows][kTiles];
      if (kTeams == 1 || team < stages) load(it, team, next);
#pragma unroll 1
      for (int s = 0; s < stages; ++s) {
        if (kTeams > 1 && s % kTeams != team) {  // another team's
          if (kScaleBufs < kStages) {
            if (lead == kScaleBufs)
              back.next();
            else
              ++lead;
          }
          ring.next();
          sring.next();
          continue;
        }
        // rows' columns: [tile][128 rows][4]
        uint32_t x[kRowTiles * 4];
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
          for (int i = 0; i < kRowTiles / kTiles * 4; ++i)
            x[j * (kRowTiles / kTiles * 4) + i] = i < kRows ? next[i][j] : 0u;
        if (s + kTeams < stages) load(it, s + kTeams, next);
        // The instructions that read this buffer must have completed: with a
        // buffer for each stage, they had before the stage was filled again.
        const auto filled = [&] {
          return wait_all(b.full + 8 * ring.st, ring.phase, abort_flag,
                          a.status);
        };
        if (kScaleBufs == kStages) {
          if (!filled()) return false;
        } else if (lead == kScaleBufs) {
          if (!wait_all(b.empty + 8 * back.st, back.phase, abort_flag,
                        a.status))
            return false;
          back.next();
        } else {
          ++lead;
        }
        tc::tc_fence_after();
        tmem_st(out + sring.st * kScales + kScaleX, x);
        if (kScaleBufs < kStages && !filled()) return false;
        const uint32_t from = sb + ring.st * kStage + kCodeBytes + lane * 16;
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
          uint32_t w[kScaleA];
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            const uint4 v = lds16(from + m * kRec + j * kScaleTile);
            w[4 * j] = v.x, w[4 * j + 1] = v.y;
            w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
          }
          tmem_st(out + sring.st * kScales + m * kScaleA, w);
        }
        tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(b.scales + 8 * sring.st);
        ring.next();
        sring.next();
      }
      return true;
    });
  }

  // ---- the matrix instructions.  The whole warp runs the loop and one lane
  // issues: the operands then are uniform.
  __device__ static void multiply(const GmmArgs& a, uint32_t sb,
                                  const Bars& b, const int2* chunks,
                                  int n_items, int tiles, uint32_t tmem,
                                  int lane, volatile int* abort_flag) {
    const int stages = a.l.stages();
    if (PAIR && rank() != 0) return;  // the first CTA's issues for both
    const bool leader = lane == 0;
    Ring<> ring;
    Ring<kScaleBufs> sring;
    int buf = 0;
    uint32_t acc_phase = 1;
    passes(a, chunks, n_items, tiles, [&](const Item& it) {
      const uint32_t idesc =
          idesc_mx(BLOCK, kTileN * kCtas, columns(it.rows));
      const uint32_t d = tmem + buf * kAcc;
      if (!wait_all(b.acc_empty + 8 * buf, acc_phase, abort_flag, a.status))
        return false;
#pragma unroll 1
      for (int s = 0; s < stages; ++s) {
        if (!wait_all(b.full + 8 * ring.st, ring.phase, abort_flag,
                      a.status) ||
            !wait_all(b.scales + 8 * sring.st, sring.phase, abort_flag,
                      a.status))
          return false;
        tc::tc_fence_after();
        const uint32_t at = sb + ring.st * kStage;
        const uint32_t sa = tmem + kScaleAt + sring.st * kScales;
        const uint32_t sx = sa + kScaleX;
        const uint64_t ad = tc::smem_desc(at, 16, 1024);
        const uint64_t bd = tc::smem_desc(at + kX, 16, 1024);
        const int steps = (a.l.K - s * kStageK + 63) / 64;
        if (leader) {
#pragma unroll
          for (int k = 0; k < kStageK / 64; ++k) {
            if (k >= steps) break;
            // four scales of 16 are a word's, two of 32 half of one
            const int tile = BLOCK == 16 ? k : k / 2;
            const uint32_t id =
                BLOCK == 16 ? 0u : (k & 1) * (2u << 4 | 2u << 29);
#pragma unroll
            for (int m = 0; m < kMats; ++m) {
              const uint64_t am = ad + ((m * kRec >> 4) + 2 * k);
              const uint32_t sm = sa + m * kScaleA + 4 * tile;
              const uint32_t st = sx + tile * (kRowTiles / kTiles * 4);
              if (PAIR)
                umma_mx_pair<BLOCK>(d + m * NT, am, bd + 2 * k, idesc | id,
                                    sm, st, s > 0 || k > 0);
              else
                umma_mx<BLOCK>(d + m * NT, am, bd + 2 * k, idesc | id, sm, st,
                               s > 0 || k > 0);
            }
          }
          commit(b.empty + 8 * ring.st);
        }
        __syncwarp();
        ring.next();
        sring.next();
      }
      if (leader) commit(b.acc_full + 8 * buf);
      __syncwarp();
      if (++buf == kBuffers) {
        buf = 0;
        acc_phase ^= 1;
      }
      return true;
    });
    // drain: every instruction that this warp issued
    if (leader) {
      if (PAIR)
        tc::umma_commit_pair(b.done);
      else
        tc::umma_commit(b.done);
      tc::mbar_wait(b.done, 0, nullptr, a.status);
    }
  }
  // Arrives on a barrier of the CTA that issues.  What it tells of is in
  // tensor memory or was brought by copies, and complete; so nothing waits for
  // a release to the whole cluster, which takes longer than a stage (gate and
  // up of 32768 rows, at that step: 727 us with it, 612 without).
  __device__ static __forceinline__ void arrive(uint32_t bar) {
    if (PAIR)
      asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                       tc::map_to_rank(bar, 0))
                   : "memory");
    else
      tc::mbar_arrive(bar);
  }
  // Arrives, in both CTAs of a pair, when all instructions so far are done.
  __device__ static __forceinline__ void commit(uint32_t bar) {
    if (PAIR)
      tc::umma_commit_pair_mc(bar);
    else
      tc::umma_commit(bar);
  }
  // ---- sums to rows of the output, a thread a column of the weights
  __device__ static void write_out(const GmmArgs& a, const Bars& b,
                                   const int2* chunks, int n_items, int tiles,
                                   uint32_t tmem, int warp, int lane,
                                   volatile int* abort_flag) {
    int buf = 0;
    uint32_t phase = 0;
    launch::wait_for_previous();
    passes(a, chunks, n_items, tiles, [&](const Item& it) {
      const Scales t = scales_of(a, it.expert);
      if (!wait_all(b.acc_full + 8 * buf, phase, abort_flag, a.status))
        return false;
      tc::tc_fence_after();
      const int quarter = warp & 3;
      const int col0 = it.tile * kTileN + quarter * 32;
      const uint32_t at =
          tmem + buf * kAcc + (static_cast<uint32_t>(quarter * 32) << 16);
      if (col0 < a.l.N) {  // N is a multiple of 32
        if constexpr (DUAL && PAIR) {
          // h of this warp's rows, then the sums are free, then the codes
          constexpr int kRows = NT / kRowParts;
          static_assert(kRows % 16 == 0, "whole loads");
          const int r0 = warp / 4 * kRows;
          float h[kRows];
#pragma unroll
          for (int r = 0; r < kRows; r += 16)
            if (r0 + r < it.rows) {
              uint32_t g[16], u[16];
              tmem_ld16(at + r0 + r, g);
              tmem_ld16(at + NT + r0 + r, u);
              tmem_ld_wait(g);
              tmem_ld_wait(u);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                h[r + i] =
                    swiglu(__uint_as_float(g[i]), __uint_as_float(u[i]), t);
            }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive(b.acc_empty + 8 * buf);
#pragma unroll
          for (int r = 0; r < kRows; r += 8)
            if (r0 + r < it.rows) write_h(a, it, col0, r0 + r, lane, h + r);
        } else {
          const int r1 = min(it.rows, (warp / 4 + 1) * (NT / kRowParts));
          if (!DUAL && BLOCK == 16 && t.first != 1.0f)
            multiply_sums(at, warp / 4 * (NT / kRowParts), r1, t.first);
#pragma unroll 1
          for (int r = warp / 4 * (NT / kRowParts); r < r1; r += 16) {
            uint32_t g[16], u[16];
            tmem_ld16(at + r, g);
            if (DUAL) tmem_ld16(at + NT + r, u);
            tmem_ld_wait(g);
            if (DUAL) {
              tmem_ld_wait(u);
#pragma unroll
              for (int i = 0; i < 16; i += 8)
                if (r + i < it.rows) {
                  float h[8];
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    h[j] = swiglu(__uint_as_float(g[i + j]),
                                  __uint_as_float(u[i + j]), t);
                  write_h(a, it, col0, r + i, lane, h);
                }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (r + i >= it.rows) break;
                const long long o =
                    static_cast<long long>(it.row + r + i) * a.l.N + col0 +
                    lane;
                const float v = t.last * __uint_as_float(g[i]);
                if (a.f32)
                  put(static_cast<float*>(a.y) + o, v);
                else
                  put(static_cast<__nv_bfloat16*>(a.y) + o, v);
              }
            }
          }
        }
      }
      if (!(DUAL && PAIR && col0 < a.l.N)) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(b.acc_empty + 8 * buf);
      }
      if (++buf == kBuffers) {
        buf = 0;
        phase ^= 1;
      }
      return true;
    });
  }

  // What sums are multiplied by: the tensor scales of the rows and the matrices,
  // up's sums by the reciprocal of h's scale too (one rounding of h less).  Down:
  // by `first`, if it is not 1, then by `last`.  Gate and up: gate's by `first`
  // and up's by `last`, whose product alone counts, and gate's by `exponent`,
  // -log2 e in it, for the exponential.
  struct Scales {
    float first, last, exponent;
  };
  static constexpr float kMinusLog2e = -1.44269504f;
  __device__ static __forceinline__ Scales scales_of(const GmmArgs& a,
                                                     int expert) {
    if (BLOCK == 32) return {1.0f, 1.0f, kMinusLog2e};
    const float x = a.x_scale, w0 = a.s0 ? a.s0[expert] : 1.0f;
    const float p0 = x * w0;
    if (!DUAL) {
      if (in_range(p0)) return {1.0f, p0, 0.0f};
      // first the scale that leads away from the end of float32's range
      const bool w_first = (p0 >= 1.0f) == (x > w0);
      return {w_first ? w0 : x, w_first ? x : w0, 0.0f};
    }
    const float w1 = a.s1 ? a.s1[expert] : 1.0f;
    const float p1 = x * w1, q1 = p1 * a.inv_out;
    if (in_range(p0) && in_range(p1) && in_range(q1))
      return {p0, q1, p0 * kMinusLog2e};
    return far_scales(x, w0, w1, a.inv_out);
  }
  // Whether a product of scales, and any sum under it, is a normal number: a sum
  // of 2^20 products of two codes and two scales of 448 at most is below 8e12,
  // and none but 0 is below 2^-20.
  __device__ static __forceinline__ bool in_range(float t) {
    return t >= 1e-25f && t <= 1e25f;
  }
  // Down's sums of rows r0 .. r1, in tensor memory, times f, before they are read
  // (a second factor where they are read took 32768 rows 348 us, not 338).
  __device__ static __noinline__ void multiply_sums(uint32_t at, int r0,
                                                    int r1, float f) {
#pragma unroll 1
    for (int r = r0; r < r1; r += 16) {
      uint32_t v[16];
      tmem_ld16(at + r, v);
      tmem_ld_wait(v);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
      tmem_st(at + r, v);
    }
    tmem_st_wait();
  }
  // Gate's and up's where one is not: the product of all in two parts of like
  // size, so that neither leaves the range before h does.  (A gate's scale over
  // 1e30 puts any sum but 0 so far out that the exponential is 0 or infinite.)
  __device__ static __noinline__ Scales far_scales(float x, float w0, float w1,
                                                   float inv_out) {
    int ex, e0, e1, eo;
    const float fx = frexpf(x, &ex);
    const float f = fx * fx * frexpf(w0, &e0) * frexpf(w1, &e1) *
                    frexpf(inv_out, &eo);
    const int e = max(-250, min(250, 2 * ex + e0 + e1 + eo)), half = e / 2;
    return {ldexpf(f, half), ldexpf(1.0f, e - half),
            fminf(x * w0, 1e30f) * kMinusLog2e};
  }
  // silu(g) u under their scales, silu(z) = z / (1 + exp(-z)); exp(-z) may be
  // infinite.
  __device__ static __forceinline__ float swiglu(float g, float u,
                                                 const Scales& t) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * t.exponent));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return t.first * g * s * (t.last * u);
  }

  // Eight rows of 32 columns of h: each lane has one column of all rows, a
  // block is the warp's lanes or half of them.
  __device__ static __forceinline__ void write_h(const GmmArgs& a,
                                                 const Item& it, int col0,
                                                 int r, int lane,
                                                 const float* h) {
    // The largest magnitudes of eight rows, each over the block's lanes: pairs of
    // lanes share out the rows and halve them, until lane % 8 has its row's.
    float q[8];
    uint32_t part[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = h[i];
      part[i] = __float_as_uint(q[i]) & 0x7fffffffu;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
#pragma unroll
      for (int i = 0; i < 4 / o; ++i) {
        const uint32_t even = part[2 * i], odd = part[2 * i + 1];
        const uint32_t other =
            __shfl_xor_sync(0xffffffffu, lane & o ? even : odd, o);
        part[i] = max(lane & o ? odd : even, other);
      }
    uint32_t most = part[0];
#pragma unroll
    for (int o = 8; o < BLOCK; o <<= 1)
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    // each scale once, then to its block's lanes
    const Block own = block_scale<BLOCK>(most);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      Block b;
      const int from = (lane & 16) + i;
      b.inv = __shfl_sync(0xffffffffu, own.inv, from);
      b.s = BLOCK == 16 ? __shfl_sync(0xffffffffu, own.s, from) : 0.0f;
      q[i] = over_scale<BLOCK>(q[i], b);
    }
    // The codes of a column's eight rows are a word; words of eight rows by
    // eight columns turn within eight lanes, halves, then bytes, then fours.
    uint32_t w = encode8(q);
    uint32_t p = __shfl_xor_sync(0xffffffffu, w, 4);
    w = lane & 4 ? __byte_perm(w, p, 0x3276) : __byte_perm(w, p, 0x5410);
    p = __shfl_xor_sync(0xffffffffu, w, 2);
    w = lane & 2 ? __byte_perm(w, p, 0x3715) : __byte_perm(w, p, 0x6240);
    p = __shfl_xor_sync(0xffffffffu, w, 1);
    w = lane & 1 ? (w & 0xf0f0f0f0u) | (p >> 4 & 0x0f0f0f0fu)
                 : (w & 0x0f0f0f0fu) | (p & 0x0f0f0f0fu) << 4;
    const int i = r + (lane & 7);
    if (i >= it.rows) return;
    const long long row = it.row + i;
    const int col = col0 + (lane & 24);
    *reinterpret_cast<uint32_t*>(a.h_codes + row * (a.l.N / 2) + col / 2) = w;
    if ((lane & (BLOCK == 32 ? 24 : 8)) == 0)
      a.h_scales[row_scale_at(BLOCK, a.rows, row, col / BLOCK)] =
          static_cast<uint8_t>(own.byte);
  }
};

template <bool DUAL, int BLOCK, int NT>
__global__ void __launch_bounds__(Gmm<DUAL, BLOCK, NT, false>::kThreads, 1)
    gmm_mx_kernel(const GmmArgs a, const __grid_constant__ CUtensorMap map) {
  Gmm<DUAL, BLOCK, NT, false>::run(a, &map);
}
template <bool DUAL, int BLOCK, int NT>
__global__ void __cluster_dims__(2, 1, 1) 
    __launch_bounds__(Gmm<DUAL, BLOCK, NT, true>::kThreads, 1)
    gmm_mx_pair_kernel(const GmmArgs a,
                       const __grid_constant__ CUtensorMap map) {
  Gmm<DUAL, BLOCK, NT, true>::run(a, &map);
}

template <bool DUAL, int BLOCK, int NT, bool PAIR>
constexpr auto kernel_of() {
  if constexpr (PAIR)
    return gmm_mx_pair_kernel<DUAL, BLOCK, NT>;
  else
    return gmm_mx_kernel<DUAL, BLOCK, NT>;
}

// Rows of codes [rows, K/2], `box` rows of 128 bytes at a time.
inline bool make_code_map(CUtensorMap* m, const void* base, int K,
                          int64_t rows, int box_rows) {
  tc::EncodeTiled fn = tc::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool DUAL, int BLOCK, int NT, bool PAIR>
cudaError_t launch_one(GmmArgs a, const void* codes, cudaStream_t s) {
  using Ker = Gmm<DUAL, BLOCK, NT, PAIR>;
  // Chunks of as few passes of NT rows as leave at most kMaxSplits more than
  // there are groups.
  const long long most = static_cast<long long>(NT) * kMaxSplits;
  a.chunk = NT * static_cast<int>((a.rows + most - 1) / most);
  a.chunks = std::min(a.n_groups, a.rows) + a.rows / a.chunk;
  static_assert(Ker::shared_bytes(kMaxChunks) <= kMaxShared,
                "any call's shared memory fits a CTA");
  Device d;
  cudaError_t e = launch::device(&d);
  if (e != cudaSuccess) return e;
  constexpr auto kernel = kernel_of<DUAL, BLOCK, NT, PAIR>();
  if ((e = launch::allow_shared<kernel>(d)) != cudaSuccess) return e;
  CUtensorMap map;
  if (!make_code_map(&map, codes, a.l.K, a.rows, Ker::kRowBox))
    return cudaErrorInvalidValue;
  const long long items =
      static_cast<long long>((a.l.tiles_n() + Ker::kCtas - 1) / Ker::kCtas) *
      a.chunks;
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>(items, d.sms / Ker::kCtas) * Ker::kCtas);
  const int bytes = Ker::shared_bytes(a.chunks);
  return launch::overlapping(kernel, grid, Ker::kThreads, bytes, s, a, map);
}

}  // namespace mx
}  // namespace moe
