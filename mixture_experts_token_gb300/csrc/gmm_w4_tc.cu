// Products of many bf16 rows with 4-bit expert weights on tcgen05.
//
// The matrix instructions of gmm_w4.cuh take eight rows at a time, nine
// clocks each, so past about a dozen rows a group they, and not the weights'
// bytes, set the time.  Here the weights are the M = 128 operand and up to
// 48 rows of x the N operand of tcgen05.mma:
//
// * Sixteen warps expand codes to bf16 (exactly code - zero, see expand()) and
//   store them to tensor memory as the A operand: what shared memory would
//   have to take and give again, four bytes for each byte of codes, is twice
//   its bandwidth at the rate HBM delivers codes.  A lane's words are in the
//   order of the 16x128b store, so nothing is shuffled.
// * Two warps, one for each tile, issue the matrix instructions, a group of
//   rows of W at a time into one of two partial accumulators.
// * Eight warps, a thread per column of W, add scale * partial in float32
//   registers while the next group runs, and at the end write the rows.
// * One thread brings x by TMA (rows past the group are other groups' rows
//   and columns past K zeros; neither reaches a row that is written).
//
// A CTA per SM walks over items: 128 columns of the gate and the up matrix,
// or 256 of the down matrix, and 48 rows of one group.  Every wait is bounded;
// one that gives up raises MOE_DEV_TIMEOUT and the CTA drains and returns.
//
// Measured, 7168 x 2048 experts, groups of 128: 1024 tokens over 256 experts
// (32 rows each) 2.3 ms, of which its bytes need 39% at 6.8 TB/s; 256 tokens
// over 32 experts (64 rows each) 602 us.  A tile of 64 rows of W takes about
// 1000 clocks whatever the rows, and no one unit bounds it: without the matrix
// instructions, the tensor memory traffic, the expansion or the copies of x,
// one at a time, it stays within 10% of that, and with all of them gone 560
// clocks are left.  Hand-overs are not what is left: stages of twice the rows
// halved them and changed nothing (339 us both, 128 tokens of 32 experts).
// Each role's warp has about 150 dependent instructions a tile, 7 warps share
// a scheduler, and 864 threads leave each 72 registers, in which the adding
// warps do not fit (52 to 88 bytes a thread spilled) and wait for the six
// loads of a partial sum in turn.
#include <atomic>

#include "gmm_w4.cuh"

namespace moe {
namespace tc {
// The GEMMs' test hook (gmm_tc.cu): stop the producer after this many stage
// fills (-1: never), so that the next wait runs out.
extern std::atomic<long long> g_stall_after_fills;
}  // namespace tc

namespace w4 {
namespace {

using tc::fence_barrier_init;
using tc::mbar_arrive;
using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::smem_desc;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::umma_commit;

constexpr int kNR = 48;            // rows of a pass
// Warps that expand: tile w / 4 % 2, lanes 32 (w % 4).., and the first or the
// second 64 rows of W of every stage (w / 8).
constexpr int kExpandWarps = 16;
constexpr int kAddWarps = 8;       // tile w / 4, lanes 32 (w % 4)..
constexpr int kMmaWarp = kExpandWarps + kAddWarps;  // one for each tile
constexpr int kCopyWarp = kMmaWarp + 2;
constexpr int kTcWarps = kCopyWarp + 1;
constexpr int kTcThreads = kTcWarps * 32;
constexpr int kStageK = 128;       // rows of W in a stage: two tiles
constexpr int kStages = 2;
constexpr int kXStages = 4;        // further ahead: x comes from L2 or HBM
constexpr int kXBytes = kNR * 128;  // 64 columns of x
// Tiles of codes, with their zero points, that each warp has in flight.
constexpr int kCodeTiles = 4;
constexpr int kTmemA = 256;        // columns: accumulators, then A
constexpr int kSumPitch = kNR + 1;
constexpr unsigned kSleepNs = 100;

struct TcArgs {
  const int32_t *offsets, *map;
  const char *w0, *w1;
  __nv_bfloat16* out;
  int32_t* status;
  Layout l;
  int n_experts, n_groups, rows, chunk, chunks;
  long long stall_after_fills;  // tests of the timeout path only (-1: off)
};

// Shared memory, from a 1024-byte boundary.
struct TcSmem {
  int codes, zeros, sums, bars, groups, total;
};
__host__ __device__ constexpr TcSmem tc_smem(const Layout& l, int chunks) {
  TcSmem m = {};
  m.codes = kXStages * 2 * kXBytes;
  m.zeros = m.codes + kExpandWarps * kCodeTiles * 2 * kTileBytes;
  m.sums = m.zeros + (l.zeros ? kExpandWarps * kCodeTiles * 2 * 16 *
                                    (kStepK / l.group)
                              : 0);
  m.bars = m.sums + 128 * kSumPitch * 4;
  m.groups = m.bars + 512;
  m.total = m.groups + 8 * chunks;
  return m;
}
static_assert(tc_smem({0, 0, 32, true}, kMaxChunks).total + 1024 <=
                  kMaxShared,
              "any call's shared memory fits a CTA");

// D (+)= A B over N16 * 16 of k, with A in tensor memory (8 columns for each
// 16 of k) and B in shared memory (32 bytes, 2 in the descriptor); `leader`
// in one lane of the warp.  The whole warp runs the loop around it: the
// operands then are uniform, and need not be moved from one lane's registers
// for every instruction.
template <int N16>
__device__ __forceinline__ void umma_ts(bool leader, uint32_t d, uint32_t a,
                                        uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  if (!leader) return;
  if (N16 == 4)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 a1, a2, a3;\n\t"
        ".reg .b64 b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, %4, %4;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\t"
        "add.u32 a3, %1, 24;\n\tadd.u64 b1, %2, 2;\n\t"
        "add.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, q;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, q;\n\t}\n" ::
            "r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, %4, %4;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u64 b1, %2, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t}\n" ::
            "r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit(bool leader, uint32_t bar) {
  if (leader) umma_commit(bar);
}

// 16 lanes x 32 columns: four words' operands in order.
__device__ __forceinline__ void tmem_st_operands(uint32_t at,
                                                 const uint32_t (&r)[4][4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, "
      "%7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(r[0][0]), "r"(r[0][1]), "r"(r[0][2]), "r"(r[0][3]), "r"(r[1][0]),
      "r"(r[1][1]), "r"(r[1][2]), "r"(r[1][3]), "r"(r[2][0]), "r"(r[2][1]),
      "r"(r[2][2]), "r"(r[2][3]), "r"(r[3][0]), "r"(r[3][1]), "r"(r[3][2]),
      "r"(r[3][3])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, "
      "%7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(at)
      : "memory");
}

// Sleeps between looks, so that the many warps that wait leave the issue
// slots and the shared-memory pipe to those that work.
static __device__ __noinline__ bool wait_asleep(uint32_t bar, uint32_t phase,
                                                volatile int* abort_flag,
                                                int32_t* status) {
  const uint64_t t0 = tc::globaltimer();
  uint32_t looks = 0;
  while (true) {
    __nanosleep(kSleepNs);
    if (tc::mbar_try_wait(bar, phase)) return true;
    if ((++looks & 15u) == 0) {
      if (*abort_flag) return false;
      if (tc::globaltimer() - t0 > tc::kWaitLimitNs) {
        *abort_flag = 1;
        if (status) atomicOr(status, MOE_DEV_TIMEOUT);
        return false;
      }
    }
  }
}
// The first look is inline: a call costs several hundred clocks here.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t phase,
                                         volatile int* abort_flag,
                                         int32_t* status) {
  return tc::mbar_try_wait(bar, phase) ||
         wait_asleep(bar, phase, abort_flag, status);
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t phase,
                                         volatile int* abort_flag,
                                         int32_t* status) {
  return __all_sync(0xffffffffu, wait_one(bar, phase, abort_flag, status));
}

// A look ahead at a barrier, without waiting: asked before other work, its
// answer is there after it.
__device__ __forceinline__ bool ready(uint32_t bar, uint32_t phase) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(phase)
      : "memory");
  return ok != 0;
}

template <bool DUAL, int G, bool Z>
struct TcKernel {
  static constexpr int E = kStepK / G;
  static constexpr int kChunk =
      kTiles * kTileBytes + 8 * E * (Z ? 6 : 4);  // bytes of a whole step
  static constexpr int kCols = DUAL ? 128 : 256;  // of an item

  // Shared-memory addresses.  A stage is full when both tiles' codes are
  // there, and empty when both tiles' instructions have read it; the same for
  // x; partial sums have two buffers for each tile.
  struct Bars {
    uint32_t full, empty, x_full, x_empty, p_full, p_empty, done;
  };
  // Where record `i` (0..7) of tile m of an item starts.  One past the last
  // is the last again: its columns are not written.
  __device__ static const char* record(const TcArgs& a, int ex, int nb, int m,
                                       int i) {
    const int rec = DUAL ? nb * 8 + i : nb * 16 + m * 8 + i;
    return (DUAL && m == 1 ? a.w1 : a.w0) + ex * a.l.matrix() +
           min(rec, a.l.tiles_n() - 1) * a.l.record();
  }

  // Calls f(item's column block, expert, first row, end of rows) for every
  // pass of this CTA until it returns false.
  template <typename F>
  __device__ static void passes(const TcArgs& a, const int2* chunks,
                                int n_items, int blocks, const F& f) {
#pragma unroll 1
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
      const int2 c = chunks[item / blocks];
      const int ex = a.map ? a.map[c.x] : c.x;
      const int r1 = chunk_end(a, c);
#pragma unroll 1
      for (int row = c.y; row < r1; row += kNR)
        if (!f(item % blocks, ex, row, r1)) return;
    }
  }

  __device__ static void run(const TcArgs& a, const CUtensorMap* map) {
    extern __shared__ __align__(1024) char raw[];
    char* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    __shared__ int abort_word;
    __shared__ uint32_t tmem_word;
    volatile int* abort_flag = &abort_word;
    const TcSmem m = tc_smem(a.l, a.chunks);
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const uint32_t sb = smem_u32(base);
    Bars b;
    b.full = sb + m.bars;
    b.empty = b.full + 8 * kStages;
    b.x_full = b.empty + 8 * kStages;
    b.x_empty = b.x_full + 8 * kXStages;
    b.p_full = b.x_empty + 8 * kXStages;
    b.p_empty = b.p_full + 32;
    b.done = b.p_empty + 32;
    if (threadIdx.x == 0) {
      abort_word = 0;
      for (int i = 0; i < kStages; ++i) {
        mbar_init(b.full + 8 * i, kExpandWarps);
        mbar_init(b.empty + 8 * i, 2);
      }
      for (int i = 0; i < kXStages; ++i) {
        mbar_init(b.x_full + 8 * i, 1);
        mbar_init(b.x_empty + 8 * i, 2);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(b.p_full + 8 * i, 1);
        mbar_init(b.p_empty + 8 * i, kAddWarps / 2);
      }
      mbar_init(b.done, 1);
      mbar_init(b.done + 8, 1);
      fence_barrier_init();
      tc::fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
      tc::tmem_alloc(smem_u32(&tmem_word), tc::kTmemCols);
      tc::tmem_relinquish();
    }
    int2* chunks = reinterpret_cast<int2*>(base + m.groups);
    const int n_chunks = find_chunks<kTcWarps>(a, chunks);  // barriers within
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_word;
    const int blocks = (a.l.N + kCols - 1) / kCols;
    const int n_items = n_chunks * blocks;
    if (warp < kExpandWarps)
      expand_codes(a, m, sb, b, chunks, n_items, blocks, tmem, warp, lane,
                   abort_flag);
    else if (warp < kExpandWarps + kAddWarps)
      add_parts(a, reinterpret_cast<float*>(base + m.sums), b, chunks,
                n_items, blocks, tmem, warp - kExpandWarps, lane, abort_flag);
    else if (warp < kCopyWarp)
      multiply(a, sb, b, chunks, n_items, blocks, tmem, warp - kMmaWarp, lane,
               abort_flag);
    else
      copy_rows(a, map, sb, b, chunks, n_items, blocks, lane, abort_flag);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, tc::kTmemCols);
  }

  // ---- codes to operands: two records of a tile of 64 rows at a time
  __device__ static void expand_codes(const TcArgs& a, const TcSmem& m,
                                      uint32_t sb, const Bars& b,
                                      const int2* chunks, int n_items,
                                      int blocks, uint32_t tmem, int warp,
                                      int lane, volatile int* abort_flag) {
    const int tiles_k = a.l.tiles_k(), t = warp / 4 % 2, q = warp % 4;
    const int c = lane >> 2, turn = warp / 8;  // tile of a stage
    const uint32_t codes =
        sb + m.codes + warp * (kCodeTiles * 2 * kTileBytes) + lane * 16;
    const uint32_t zeros = sb + m.zeros + warp * (kCodeTiles * 2 * 16 * E);
    const uint32_t a_at = tmem + kTmemA + t * 128 +
                          (static_cast<uint32_t>(32 * q) << 16);
    // the copying side, kCodeTiles tiles ahead
    int item = blockIdx.x, row = 0, r1 = 0, tile = 0;
    const char *p0 = nullptr, *p1 = nullptr, *s0 = nullptr, *s1 = nullptr;
    const auto enter = [&] {
      const int2 chunk = chunks[item / blocks];
      const int ex = a.map ? a.map[chunk.x] : chunk.x;
      row = chunk.y;
      r1 = chunk_end(a, chunk);
      s0 = record(a, ex, item % blocks, t, 2 * q) + lane * 16;
      s1 = record(a, ex, item % blocks, t, 2 * q + 1) + lane * 16;
    };
    const auto rewind = [&] {  // to this set's first tile of a pass
      tile = turn;
      p0 = s0 + tile * kTileBytes;
      p1 = s1 + tile * kTileBytes;
    };
    const auto next_pass = [&] {
      row += kNR;
      if (row >= r1) {
        item += gridDim.x;
        if (item < n_items) enter();
      }
      rewind();
    };
    if (item < n_items) {
      enter();
      rewind();
      while (tile >= tiles_k && item < n_items) next_pass();
    }
    int in_slot = 0;
    const auto copy_tile = [&] {
      if (item < n_items) {
        const uint32_t dst = codes + in_slot * (2 * kTileBytes);
        copy16(dst, p0);
        copy16(dst + kTileBytes, p1);
        if (Z && lane < E) {  // the step's zero points, 16 E bytes
          const int at = tile % kTiles;  // the pointers are at this tile
          const int to = (min(tiles_k - tile + at, kTiles) - at) * kTileBytes +
                         32 * E;
          const uint32_t d = zeros + in_slot * (2 * 16 * E) + lane * 16;
          copy16(d, p0 + to);
          copy16(d + 16 * E, p1 + to);
        }
        // two tiles on, past a step's scales where they lie between
        tile += 2;
        const int skip = 2 * kTileBytes + (tile % kTiles < 2
                                               ? kChunk - kTiles * kTileBytes
                                               : 0);
        p0 += skip;
        p1 += skip;
        while (tile >= tiles_k && item < n_items) next_pass();
      }
      copies_commit();
      in_slot = in_slot == kCodeTiles - 1 ? 0 : in_slot + 1;
    };
#pragma unroll 1
    for (int i = 0; i < kCodeTiles; ++i) copy_tile();

    int slot = 0, st = 0;
    uint32_t phase = 1;
    passes(a, chunks, n_items, blocks, [&](int, int, int, int) {
      uint32_t z[2][2];
      z[0][0] = z[0][1] = z[1][0] = z[1][1] = 0xbe00be00u;  // -8/64
#pragma unroll 1
      for (int k = turn; k < tiles_k + turn; k += 2) {
        uint32_t op[2][4][4];
        const bool here = k < tiles_k;  // else the stage has one tile
        if (here) {
          copies_wait<kCodeTiles - 1>();
          if (Z) __syncwarp();
          uint32_t w[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint4 v =
                lds16(codes + slot * (2 * kTileBytes) + r * kTileBytes);
            w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (Z && (h == 0 || G == 32)) {
                const int g = (k % kTiles * kTileK + 32 * h) / G;
                const uint32_t v = lds2(zeros + slot * (2 * 16 * E) +
                                        r * 16 * E + (c * E + g) * 2);
                constexpr uint32_t kMinus = kPow127 | 0x80008000u;
                z[r][0] = fma2(__byte_perm(v, 0, 0x4040), kMinus, 0);
                z[r][1] = fma2(__byte_perm(v, 0, 0x4141), kMinus, 0);
              }
              expand(w[r][2 * h], z[r], op[r][2 * h]);
              expand(w[r][2 * h + 1], z[r], op[r][2 * h + 1]);
            }
          }
          if (Z) __syncwarp();  // every lane has read what is copied over
          copy_tile();
          slot = slot == kCodeTiles - 1 ? 0 : slot + 1;
        }
        if (!wait_all(b.empty + 8 * st, phase, abort_flag, a.status))
          return false;
        if (here) {
          tc_fence_after();
          const uint32_t at = a_at + st * 64 + turn * 32;
          tmem_st_operands(at, op[0]);
          tmem_st_operands(at + (16u << 16), op[1]);
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b.full + 8 * st);
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
      }
      return true;
    });
    copies_wait<0>();
  }

  // ---- rows of x by TMA: 64 columns of the pass's rows at a time
  __device__ static void copy_rows(const TcArgs& a, const CUtensorMap* map,
                                   uint32_t sb, const Bars& b,
                                   const int2* chunks, int n_items,
                                   int blocks, int lane,
                                   volatile int* abort_flag) {
    if (lane != 0) return;
    const int tiles_k = a.l.tiles_k();
    int xs = 0;
    long long filled = 0;
    uint32_t phase = 1;
    passes(a, chunks, n_items, blocks, [&](int, int, int row, int) {
#pragma unroll 1
      for (int k = 0; k < tiles_k; k += 2) {
        if ((a.stall_after_fills >= 0 && filled >= a.stall_after_fills) ||
            !wait_one(b.x_empty + 8 * xs, phase, abort_flag, a.status))
          return false;
        const int n = min(2, tiles_k - k);
        mbar_expect_tx(b.x_full + 8 * xs, n * kXBytes);
        for (int i = 0; i < n; ++i)
          tc::tma_load_2d(sb + (2 * xs + i) * kXBytes, map,
                          b.x_full + 8 * xs, (k + i) * kTileK, row);
        ++filled;
        if (++xs == kXStages) {
          xs = 0;
          phase ^= 1;
        }
      }
      return true;
    });
    // This thread's last copies must have landed before the CTA ends.  The
    // instructions that read them wait for them, unless a wait of any warp
    // gave up: also after this thread's last fill.
    for (long long i = 0; i < filled && i < kXStages; ++i) {
      if (--xs < 0) {
        xs = kXStages - 1;
        phase ^= 1;
      }
      tc::mbar_wait(b.x_full + 8 * xs, phase ^ 1, nullptr, a.status);
    }
  }

  // ---- the matrix instructions: one partial sum for each group of W's rows
  __device__ static void multiply(const TcArgs& a, uint32_t sb, const Bars& b,
                                  const int2* chunks, int n_items,
                                  int blocks, uint32_t tmem, int t, int lane,
                                  volatile int* abort_flag) {
    const int tiles_k = a.l.tiles_k();
    const uint32_t p_full = b.p_full + 16 * t, p_empty = b.p_empty + 16 * t;
    const uint32_t d = tmem + t * 128, a_at = tmem + kTmemA + t * 128;
    const bool leader = lane == 0;
    int st = 0, xs = 0, part = 0;
    uint32_t phase = 0, x_phase = 0, p_phase = 1;
    bool full = false, x_full = false, empty = false;  // the next ones, as seen ahead
    passes(a, chunks, n_items, blocks, [&](int, int, int row, int r1) {
      const int n = (min(kNR, r1 - row) + 15) / 16 * 16;
      const uint32_t idesc =
          tc::make_idesc(128, 16, false) + ((n - 16) >> 3 << 17);
#pragma unroll 1
      for (int k = 0; k < tiles_k; k += 2) {
        if (!__all_sync(0xffffffffu, full) &&
            !wait_all(b.full + 8 * st, phase, abort_flag, a.status))
          return false;
        if (!__all_sync(0xffffffffu, x_full) &&
            !wait_all(b.x_full + 8 * xs, x_phase, abort_flag, a.status))
          return false;
        tc_fence_after();
        const int st_next = st == kStages - 1 ? 0 : st + 1;
        const uint32_t phase_next = st_next == 0 ? phase ^ 1 : phase;
        const int xs_next = xs == kXStages - 1 ? 0 : xs + 1;
        const uint32_t x_phase_next = xs_next == 0 ? x_phase ^ 1 : x_phase;
        const uint64_t bd = smem_desc(sb + xs * 2 * kXBytes, 16, 1024);
        const uint32_t at = a_at + st * 64;
        full = ready(b.full + 8 * st_next, phase_next);
        x_full = ready(b.x_full + 8 * xs_next, x_phase_next);
        constexpr int kN16 = G == 32 ? 2 : 4;  // instructions in a row
#pragma unroll
        for (int h = 0; h < kStageK / 16; h += kN16) {
          if (h >= 4 && k + 1 == tiles_k) break;  // a stage of one tile
          const bool first = h * 16 % G == 0;
          if (first) {
            if (!__all_sync(0xffffffffu, empty) &&
                !wait_all(p_empty + 8 * part, p_phase, abort_flag, a.status))
              return false;
            tc_fence_after();
          }
          // the second tile's x is a box further on
          umma_ts<kN16>(leader, d + part * 64, at + h * 8,
                        bd + (h / 4 * (kXBytes >> 4) + h % 4 * 2), idesc,
                        first ? 0u : 1u);
          if ((h + kN16) * 16 % G == 0 ||
              (h + kN16 == 4 && k + 1 == tiles_k)) {
            commit(leader, p_full + 8 * part);
            part ^= 1;
            if (part == 0) p_phase ^= 1;
            empty = ready(p_empty + 8 * part, p_phase);
          }
        }
        commit(leader, b.empty + 8 * st);
        commit(leader, b.x_empty + 8 * xs);
        xs = xs_next;
        x_phase = x_phase_next;
        st = st_next;
        phase = phase_next;
      }
      return true;
    });
    // drain: every instruction that this warp issued
    commit(leader, b.done + 8 * t);
    if (leader) tc::mbar_wait(b.done + 8 * t, 0, nullptr, a.status);
  }

  // ---- scale * partial sums, a thread per column of W, and the output
  __device__ static void add_parts(const TcArgs& a, float* sums,
                                   const Bars& b, const int2* chunks,
                                   int n_items, int blocks, uint32_t tmem,
                                   int warp, int lane,
                                   volatile int* abort_flag) {
    const int t = warp / 4, q = warp % 4;
    const int col = lane & 15, n_in = 32 * q + lane;  // column of the tile
    const int tiles_k = a.l.tiles_k();
    const int groups = (tiles_k * kTileK + G - 1) / G;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    int part = 0;
    uint32_t phase = 0;
    // After a wait that gave up the loops run on without waiting, so that
    // the warps meet at their barriers.
    bool ok = true;
    passes(a, chunks, n_items, blocks, [&](int nb, int ex, int row, int r1) {
      const int rows = min(kNR, r1 - row);
      const char* rec =
          record(a, ex, nb, t, 2 * q + (lane >> 4)) + (col & 7) * (4 * E) +
          (col >> 3) * 2;
      const auto load_scale = [&](int g) {
        const int step = g / E;
        const char* p = rec + step * kChunk +
                        min(kTiles, tiles_k - step * kTiles) * kTileBytes +
                        g % E * 4;
        return __ldg(reinterpret_cast<const unsigned short*>(p));
      };
      float acc[kNR];
#pragma unroll
      for (int i = 0; i < kNR; ++i) acc[i] = 0.0f;
      unsigned short next = load_scale(0);
#pragma unroll 1
      for (int g = 0; g < groups; ++g) {
        const float s = __uint_as_float(static_cast<uint32_t>(next) << 16);
        if (g + 1 < groups) next = load_scale(g + 1);
        if (ok)
          ok = wait_all(b.p_full + 16 * t + 8 * part, phase, abort_flag,
                        a.status);
        if (ok) {
          tc_fence_after();
          const uint32_t d = tmem + lanes + t * 128 + part * 64;
#pragma unroll
          for (int i = 0; i < kNR; i += 8) {
            if (i >= rows) break;
            uint32_t v[8];
            tmem_ld8(d + i, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[i + j] = fmaf(s, __uint_as_float(v[j]), acc[i + j]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b.p_empty + 16 * t + 8 * part);
        }
        part ^= 1;
        if (part == 0) phase ^= 1;
      }
      // the sums are 1/64 of the products
      if (DUAL) {
        if (t == 1)
#pragma unroll
          for (int i = 0; i < kNR; ++i) sums[n_in * kSumPitch + i] = acc[i];
        barrier();
        const int n = nb * 128 + n_in;
        if (t == 0 && ok && n < a.l.N) {
#pragma unroll
          for (int i = 0; i < kNR; ++i) {
            const float g = 64.0f * acc[i];
            const float u = 64.0f * sums[n_in * kSumPitch + i];
            if (i < rows)
              a.out[static_cast<long long>(row + i) * a.l.N + n] =
                  __float2bfloat16(g / (1.0f + expf(-g)) * u);
          }
        }
        barrier();
      } else {
        const int n = nb * 256 + t * 128 + n_in;
        if (ok && n < a.l.N) {
#pragma unroll
          for (int i = 0; i < kNR; ++i)
            if (i < rows)
              a.out[static_cast<long long>(row + i) * a.l.N + n] =
                  __float2bfloat16(64.0f * acc[i]);
        }
      }
      return true;
    });
  }

  __device__ static __forceinline__ void barrier() {
    asm volatile("bar.sync 1, %0;" ::"n"(kAddWarps * 32) : "memory");
  }
};

template <bool DUAL, int G, bool Z>
__global__ void __launch_bounds__(kTcThreads, 1)
    gmm_w4_tc_kernel(const TcArgs a, const __grid_constant__ CUtensorMap map) {
  TcKernel<DUAL, G, Z>::run(a, &map);
}

template <bool DUAL, int G, bool Z>
cudaError_t launch_tc(const TcArgs& a, const CUtensorMap& map,
                      const Device& d, cudaStream_t s) {
  constexpr auto kernel = gmm_w4_tc_kernel<DUAL, G, Z>;
  const cudaError_t e = launch::allow_shared<kernel>(d);
  if (e != cudaSuccess) return e;
  const int cols = TcKernel<DUAL, G, Z>::kCols;
  const long long items =
      static_cast<long long>((a.l.N + cols - 1) / cols) * a.chunks;
  const unsigned grid =
      static_cast<unsigned>(std::min<long long>(items, d.sms));
  kernel<<<grid, kTcThreads, tc_smem(a.l, a.chunks).total + 1024, s>>>(a,
                                                                        map);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gmm_w4_tc(bool dual, GmmArgs g, cudaStream_t s) {
  set_chunk(&g, kNR);
  Device d;
  cudaError_t e = launch::device(&d);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (!tc::make_map(&map, g.x, g.l.K, g.rows, kTileK, kNR))
    return cudaErrorInvalidValue;
  const TcArgs a = {g.offsets, g.map,    g.w0,        g.w1,
                    static_cast<__nv_bfloat16*>(g.out), g.status, g.l,
                    g.n_experts, g.n_groups, g.rows, g.chunk, g.chunks,
                    tc::g_stall_after_fills.load()};
#define MOE_W4_CASE(GROUP)                                                  \
  if (g.l.group == GROUP) {                                                 \
    if (dual)                                                               \
      return g.l.zeros ? launch_tc<true, GROUP, true>(a, map, d, s)         \
                       : launch_tc<true, GROUP, false>(a, map, d, s);       \
    return g.l.zeros ? launch_tc<false, GROUP, true>(a, map, d, s)          \
                     : launch_tc<false, GROUP, false>(a, map, d, s);        \
  }
  MOE_W4_CASE(32)
  MOE_W4_CASE(64)
  MOE_W4_CASE(128)
#undef MOE_W4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace w4
}  // namespace moe
