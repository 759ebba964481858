// What the kernels of linear layers share: the three products and how their
// operands lie, parameters, tiles, waits, and the epilogue.
//
// The products of a layer with weights w (out x in), for the rows of a group:
//   forward  z = x w^T        D rows x out, sums over in
//   grad_x   dz w             D rows x in,  sums over out
//   grad_w   dz^T x           D out x in,   sums over rows
// The tensor cores take operands either with the summed index contiguous (K-major) or
// with the other one (MN-major), so nothing is transposed in memory.  One operand has
// their M, 128 a CTA, the other their N, any multiple of 16.  M are D's columns and N its
// rows, so that a lane of the accumulator is a column of D, and what a warp stores at once
// lies next to each other:
//              M                              N
//   forward    outputs, w       K-major       rows, x       K-major
//   grad_x     inputs, w^T      MN-major      rows, dz      K-major
//   grad_w     inputs, x^T      MN-major      outputs, dz^T MN-major
// Groups are ragged in rows, the N of the first two: a tile of 5 rows
// costs an instruction of 16 columns, and one that ends with its group what it
// has.  (With rows as M, in steps of 128 or 256, 4096 tokens x 8 of 64 experts,
// 4096 -> 2048, took 392 us.)  The rows of the next group that its last copy of rows brings
// along are not multiplied, or end in columns of the accumulator that are not
// stored.
// grad_w has the rows in the sum, and has to keep other groups' out of it: it stops at
// the group's last 16 rows and zeroes, in shared memory, what of those is not the
// group's, in both operands (a NaN there would come through a zero in the
// other).  w is a tensor of three dimensions, so that copies past an expert's
// rows bring zeros.
#pragma once
#include <cuda.h>

#include <algorithm>

#include "linear.h"
#include "moe_common.cuh"
#include "tensor_map.cuh"

namespace gb300 {

constexpr int kLinM = 128;            // the M of a CTA: one accumulator lane each
constexpr int kLinK = 64;             // summed elements of a block: 128 bytes, a swizzle row
constexpr int kLinEpiWarps = 8;
constexpr int kLinZeroWarp = 2 + kLinEpiWarps;  // grad_w: zeroes what is no group's in a stage
constexpr int kLinNWarp = 3 + kLinEpiWarps;     // the second producer
constexpr int kLinThreads = 128 + 32 * kLinEpiWarps;
// Deeper rings begin later: all of them are asked for at once, and the first lands with the
// others (64 x 1704 x 656 with a tile of 32: 6.3 us with 8, 6.9 with 11).
constexpr int kLinMaxStages = 8;
constexpr uint32_t kLinABytes = kLinM * kLinK * 2;
constexpr uint32_t kLinChunkBytes = 64 * kLinK * 2;  // MN-major: 64 columns by 64 of the sum
constexpr uint32_t kLinBufBytes = 32 * 32 * 4;       // kSplit: 32 x 32 sums
constexpr uint32_t kLinSmemLimit = 232448;

struct LinearParams {
  uint16_t* out;             // D, rows contiguous
  uint16_t* preact;          // forward: z, or null
  const uint16_t* bias;      // forward: groups x n, or null
  const uint16_t* residual;  // forward: or null
  int64_t ldr;
  const int32_t* offsets;    // of the groups of rows; null: one group
  const float* strips;       // grad_w: sums of dz over strips of rows (linear_rows.cuh), or null
  uint16_t* grad_bias;
  int32_t strip_rows;
  int32_t rows;              // of all groups, and those of none
  int32_t m;                 // grad_w: rows of a group's D (outputs)
  int32_t n;                 // columns of D
  int32_t k;                 // forward, grad_x: length of the sums
  int32_t groups;
  int32_t tile;              // the N of a tile, at most
  int32_t tile_shift;        // forward, grad_x: its logarithm
  int32_t m_tiles, n_tiles;  // M: of a group; N: grad_w's, of a group
  int32_t box_rows;          // forward, grad_x: rows that one copy loads
  int32_t stages, split;
  int32_t activation;
  int32_t overlap;           // kOverlap*
  int32_t inject;            // 1: leave out each CTA's first loads
  int32_t error_word;
  uint64_t timeout_ns;
};

// grad_w runs beside grad_x, whose SMs it takes over as they get free (1021 x 1000 x 1411,
// with everything before: 26 us one after the other).  Both need what came before them and
// nothing of each other.  So grad_x lets grad_w start only once all of its own CTAs have
// waited for that (kOverlapFirst), grad_w begins without waiting, and waits for grad_x at
// its end (kOverlapSecond), so that what follows it follows both.
// What came before is complete when grad_x's waits return, and a CTA of grad_w starts after that.
// The instructions promise grad_x alone to see it; fences on both sides of the start carry that
// on to grad_w, whose loads of it are ordinary ones and TMA's.
enum { kOverlapNone = 0, kOverlapFirst = 1, kOverlapSecond = 2 };

__device__ __forceinline__ void linear_begin_early(const LinearParams& p) {
  if (p.overlap != kOverlapFirst) grid_launch_dependents();
}
__device__ __forceinline__ void linear_begin(const LinearParams& p) {
  if (p.overlap == kOverlapSecond) {
    __threadfence();
    fence_proxy_async_global();
    return;
  }
  grid_dependency_wait();
  if (p.overlap == kOverlapFirst) {
    __threadfence();
    grid_launch_dependents();
  }
}
__device__ __forceinline__ void linear_end(const LinearParams& p) {
  if (p.overlap == kOverlapSecond) grid_dependency_wait();
}

// MN-major operands, of M and of N
__host__ __device__ constexpr bool a_mn(int product) { return product != LINEAR_FORWARD; }
__host__ __device__ constexpr bool b_mn(int product) { return product == LINEAR_GRAD_W; }

// Shared memory past the ring: barriers, the tensor
// memory address, the abort flag, and where each group starts; 1 KiB to align.
constexpr uint32_t kLinBars = 4 * kLinMaxStages + 5;
__host__ __device__ constexpr uint32_t linear_fixed_bytes(int groups) {
  return 8 * kLinBars + 24 + 8 * (groups + 1) + 1024;
}

// ------------------------------------------------------------------ PTX
// Instruction descriptor of kind::f16: D fp32 (bits 4-5 = 1), A and B of the
// same type (bits 7-9 and 10-12: 0 fp16, 1 bf16), MN-major A and B (bits 15 and
// 16), N >> 3 in bits 17-22, M >> 4 in bits 24-28.
template <typename T, int kProduct>
__device__ __forceinline__ constexpr uint32_t linear_idesc(int m, int n) {
  return (1u << 4) | (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u) |
         (a_mn(kProduct) ? 1u << 15 : 0u) | (b_mn(kProduct) ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <bool kMn>
__device__ __forceinline__ uint64_t linear_desc(uint32_t smem_addr) {
  return kMn ? sw128_mnmajor_desc(smem_addr, kLinChunkBytes) : sw128_kmajor_desc(smem_addr);
}
// 16 of the sum further, in the descriptor's units of 16 bytes
template <bool kMn>
__device__ __forceinline__ constexpr uint32_t linear_desc_step() { return kMn ? 128u : 2u; }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Arrive on an mbarrier of the cluster without a release: it does not wait for this
// thread's stores to be performed.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// ------------------------------------------------------------------ waits
enum LinearWait : uint32_t { kLinEmpty = 1, kLinFull = 2, kLinTmemEmpty = 3, kLinTmemFull = 4,
                             kLinPeer = 5 };

// The first error of the launches on a given stream (the host maps streams to
// words); 0: none.
__device__ uint32_t g_linear_error[kErrorWords];

// Waits for phase `parity` of `bar`; gives up when the CTA does, or after the
// limit, which it records.  kCluster: for what other CTAs of the cluster wrote.
template <bool kCluster = false>
__device__ __forceinline__ bool linear_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                            uint32_t site, const LinearParams& p) {
  const auto done = [&] {
    return kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  };
  if (done()) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (done()) return true;
    if ((it & 31u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > p.timeout_ns) {
        *abort_flag = 1;
        atomicCAS(&g_linear_error[p.error_word], 0u,
                  static_cast<uint32_t>(GEMM_ERR_TIMEOUT) | (site << 8));
        return false;
      }
    }
  }
}

// The same by a whole warp: it goes on, or gives up, together.
template <bool kCluster = false>
__device__ __forceinline__ bool linear_wait_warp(uint32_t bar, uint32_t parity,
                                                 volatile int* abort_flag, uint32_t site,
                                                 const LinearParams& p) {
  return __all_sync(0xffffffffu, linear_wait<kCluster>(bar, parity, abort_flag, site, p));
}

// A wait on the way out, whether or not the CTA gave up.
__device__ __forceinline__ void linear_wait_drain(uint32_t bar, uint32_t parity,
                                                  uint64_t timeout_ns) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return;
    if ((it & 31u) == 0 && global_timer_ns() - t0 > timeout_ns) return;
  }
}

// ------------------------------------------------------------------ tiles
struct LinearTile {
  int32_t group;
  int32_t m, m_count;   // columns of D: first, and how many
  int32_t n, n_count;   // rows: forward, grad_x of all groups; grad_w of its own
  int32_t k_row;        // grad_w: the first summed row
  int32_t k_len;        // length of the sums
};

// Tiles of rows that walk over the columns together, so that what runs at once shares
// operands in L2.
constexpr int kLinRaster = 8;

// Tile t among `slow` x `fast`: bands of kLinRaster of the first, over all of the second.
__device__ __forceinline__ void linear_raster(int t, int slow, int fast, int* s, int* f) {
  if (slow == 1) {
    *s = 0;
    *f = t;
    return;
  }
  const int band = t / (kLinRaster * fast);
  const int in = t - band * kLinRaster * fast;
  const int wide = min(kLinRaster, slow - band * kLinRaster);
  *f = wide == kLinRaster ? in / kLinRaster : in / wide;
  *s = band * kLinRaster + in - *f * wide;
}

// Tiles of all groups.
template <int kProduct>
__device__ __forceinline__ int linear_tiles(const LinearParams& p, const GroupStart* start) {
  return kProduct == LINEAR_GRAD_W ? p.groups * p.m_tiles * p.n_tiles
                                   : start[p.groups].tiles * p.m_tiles;
}

// kM: the M of a tile.
template <int kProduct, int kM>
__device__ __forceinline__ LinearTile linear_tile(int t, const LinearParams& p,
                                                  const GroupStart* start) {
  LinearTile o;
  int mt, nt;
  if (kProduct == LINEAR_GRAD_W) {
    const int per = p.m_tiles * p.n_tiles;
    o.group = p.groups > 1 ? t / per : 0;
    linear_raster(t - o.group * per, p.n_tiles, p.m_tiles, &nt, &mt);
    o.n = nt * p.tile;
    o.n_count = min(p.tile, p.m - o.n);
    o.k_row = start[o.group].row;
    o.k_len = start[o.group + 1].row - o.k_row;
  } else {
    int lo = 0, hi = p.groups - 1;  // the last group with tiles * m_tiles <= t before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid].tiles * p.m_tiles <= t) lo = mid;
      else hi = mid - 1;
    }
    const int first = start[lo].row, rows = start[lo + 1].row - first;
    const int n_tiles = (rows + p.tile - 1) >> p.tile_shift;
    linear_raster(t - start[lo].tiles * p.m_tiles, n_tiles, p.m_tiles, &nt, &mt);
    // a group's tiles are of one size, to 32 rows, so that what runs at once ends at once
    const int each = n_tiles > 1 ? ((rows + n_tiles - 1) / n_tiles + 31) & ~31 : rows;
    o.group = lo;
    o.n = first + nt * each;
    o.n_count = min(each, rows - nt * each);
    o.k_row = 0;
    o.k_len = p.k;
  }
  o.m = mt * kM;
  o.m_count = min(kM, p.n - o.m);
  return o;
}

// Where each group starts, by one warp.
__device__ __forceinline__ void linear_starts(const LinearParams& p, GroupStart* start, int lane) {
  if (p.offsets) {
    find_groups(p.offsets, p.groups, start, lane, p.tile_shift);
  } else {  // one group, or none of any rows
    for (int g = lane; g <= p.groups; g += 32)
      start[g] = g ? GroupStart{(p.rows + (1 << p.tile_shift) - 1) >> p.tile_shift, p.rows}
                   : GroupStart{0, 0};
  }
}

// Whether there is anything to sum, and the tensor maps mean something.
template <int kProduct>
__device__ __forceinline__ bool linear_has_sums(const LinearParams& p) {
  return kProduct == LINEAR_GRAD_W ? p.rows > 0 : p.k > 0;
}

// Stage kb's steps of 16 along the sum.
__device__ __forceinline__ int linear_steps(const LinearTile& t, int kb) {
  return min(kLinK / 16, (t.k_len - kb * kLinK + 15) >> 4);
}
// grad_w: whether the sum ends inside a step, so that rows of the next group (or
// of none) are in it.  (Past the last row of all the copies bring zeros.)
__device__ __forceinline__ bool linear_ragged(const LinearTile& t, int kb, const LinearParams& p) {
  return p.offsets && (t.k_len & 15) && t.k_len - kb * kLinK < kLinK;
}

// Waits, in grad_w, for the last loads of ragged stages, on the way out; bit s of
// `phases` is the parity of the slot's next.
__device__ __forceinline__ void linear_drain_ragged(uint32_t first_bar, int stages, uint32_t phases,
                                                    uint64_t timeout_ns) {
  for (int s = 0; s < stages; ++s)
    linear_wait_drain(first_bar + 8u * s, ((phases >> s) & 1u) ^ 1u, timeout_ns);
}

// Zeroes, in `chunks` chunks of 64 columns, the rows of the stage's last step that
// are past the sum's end.  By a warp of its own, which is ahead of the MMAs as the
// loads are (on single CTAs with 128 columns 759 us for 4096 tokens x 8 of 64 experts
// by the MMAs' warp, 719 so); they see it after the proxy fence.
__device__ __forceinline__ void linear_zero_rows(uint32_t at, int chunks, int valid, int lane) {
  const int pieces = (((valid + 15) & ~15) - valid) * 8;
  for (int c = 0; c < chunks; ++c)
    for (int i = lane; i < pieces; i += 32)
      st_shared_v4(at + c * kLinChunkBytes + valid * 128u + i * 16u, 0, 0, 0, 0);
}

// ------------------------------------------------------------------ products of a tile
// True if the phase with the given parity has completed; does not wait.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The ring as a warp goes through it: a stage, and what its next barrier said already.
struct LinearRing {
  uint32_t bars;                 // the first of those that the warp waits on
  int stages;
  int stage;
  uint32_t phase;
  bool open;                     // the stage's has been seen to be complete

  __device__ __forceinline__ void look(uint32_t flip) { open = mbar_test_wait(bars + 8u * stage, phase ^ flip); }
  __device__ __forceinline__ void step() {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// By the whole warp: the stage's barrier, of the phase before for a producer (flip 1).
__device__ __forceinline__ bool linear_enter(const LinearRing& ring, uint32_t flip,
                                             volatile int* abort_flag, uint32_t site,
                                             const LinearParams& p) {
  return __all_sync(0xffffffffu, ring.open) ||
         linear_wait_warp(ring.bars + 8u * ring.stage, ring.phase ^ flip, abort_flag, site, p);
}

// Blocks from .. end - 1 of a tile's sum, kBlocks a stage; by a whole warp, of which one lane
// issues.  False: a wait gave up.  What bounds it with small tiles is the issuing: about 30 cycles an
// MMA (which takes 40 for an N of 32), 66 a commit, and the wait, 95; so the next stage's barrier is
// looked at before this one's MMAs are issued, whole stages have no branches, and stages have
// two blocks where there is room.
template <typename T, int kProduct, bool kPair, int kBlocks>
__device__ __forceinline__ bool linear_multiply(const LinearTile& tile, int from, int end,
                                                LinearRing& ring, uint32_t empty_bars,
                                                uint32_t ready_bars, uint32_t& ready_phase,
                                                uint32_t block_units, uint64_t a_desc0,
                                                uint64_t b_desc0, uint32_t d_tmem, uint32_t idesc,
                                                volatile int* abort_flag, const LinearParams& p) {
  constexpr uint32_t kA = linear_desc_step<a_mn(kProduct)>(), kB = linear_desc_step<b_mn(kProduct)>();
  constexpr int kSteps = kLinK / 16;
  if (from >= end) return true;
  const int left = end - from;
  const int whole = (left - 1) / kBlocks;           // stages before the last
  const auto mma = [&](uint64_t da, uint64_t db, int s, uint32_t accumulate) {
    if (kPair) umma_f16_pair(d_tmem, da + s * kA, db + s * kB, idesc, accumulate);
    else umma_f16(d_tmem, da + s * kA, db + s * kB, idesc, accumulate);
  };
  const auto commit = [&](int stage) {
    if (kPair) umma_commit_pair_mc(empty_bars + 8u * stage, 0x3);
    else umma_commit(empty_bars + 8u * stage);
  };
  ring.look(0);
  uint32_t accumulate = 0;
  for (int i = 0; i < whole; ++i) {
    if (!linear_enter(ring, 0, abort_flag, kLinFull, p)) return false;
    tc_fence_after_sync();
    const int stage = ring.stage;
    ring.step();
    ring.look(0);
    if (elect_one()) {
      const uint32_t at = stage * kBlocks * block_units;
      const uint64_t da = a_desc0 + at, db = b_desc0 + at;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          mma(da + b * block_units, db + b * block_units, s, b + s > 0 ? 1u : accumulate);
      commit(stage);
    }
    __syncwarp();
    accumulate = 1;
  }
  // the last: of fewer blocks or steps, and in grad_w ragged
  if (!linear_enter(ring, 0, abort_flag, kLinFull, p)) return false;
  const int stage = ring.stage;
  if (kProduct == LINEAR_GRAD_W && linear_ragged(tile, end - 1, p)) {
    if (!linear_wait_warp<kPair>(ready_bars + 8u * stage, (ready_phase >> stage) & 1u, abort_flag,
                                 kLinPeer, p))
      return false;
    ready_phase ^= 1u << stage;
  }
  tc_fence_after_sync();
  ring.step();
  const int steps = (left - 1 - whole * kBlocks) * kSteps + linear_steps(tile, end - 1);
  if (elect_one()) {
    const uint32_t at = stage * kBlocks * block_units;
    const uint64_t da = a_desc0 + at, db = b_desc0 + at;
    for (int s = 0; s < steps; ++s)
      mma(da + s / kSteps * block_units, db + s / kSteps * block_units, s % kSteps,
          s > 0 ? 1u : accumulate);
    commit(stage);
  }
  __syncwarp();
  return true;
}

// ------------------------------------------------------------------ loads
// What a CTA loads for each stage of a tile: of M from m on, of N from n on.
struct LinearLoads {
  int32_t m, n;
  int32_t a_boxes, b_boxes;
  uint32_t a_box_bytes, b_box_bytes, bytes;
};

// At least a box of each, also where there is nothing (past the ends they are zeros).
template <int kProduct>
__device__ __forceinline__ LinearLoads linear_loads(int m, int m_count, int n, int n_count,
                                                    const LinearParams& p) {
  LinearLoads l;
  l.m = m;
  l.n = n;
  l.a_boxes = a_mn(kProduct) ? min(max(1, (m_count + 63) >> 6), kLinM / 64) : 1;
  l.a_box_bytes = a_mn(kProduct) ? kLinChunkBytes : kLinABytes;
  l.b_boxes = max(1, b_mn(kProduct) ? (n_count + 63) >> 6 : (n_count + p.box_rows - 1) / p.box_rows);
  l.b_box_bytes = b_mn(kProduct) ? kLinChunkBytes : p.box_rows * (kLinK * 2);
  l.bytes = l.a_boxes * l.a_box_bytes + l.b_boxes * l.b_box_bytes;
  return l;
}

// A stage's operand of M, or of N, from k of the sum on, to the stage at `dst`; by one lane.
template <int kProduct, bool kPair>
__device__ __forceinline__ void linear_load_m(const LinearLoads& l, uint32_t dst, const void* tm,
                                              uint32_t full, int k, const LinearTile& t) {
  const auto load = [&](uint32_t at, int x, int y, int z) {
    if (kPair) tma_load_3d_pair(at, tm, full, x, y, z);
    else tma_load_3d(at, tm, full, x, y, z);
  };
  if (kProduct == LINEAR_FORWARD) {
    load(dst, k, l.m, t.group);
  } else {
    const int group = kProduct == LINEAR_GRAD_X ? t.group : 0;
    load(dst, l.m, t.k_row + k, group);
    if (l.a_boxes > 1) load(dst + kLinChunkBytes, l.m + 64, t.k_row + k, group);
  }
}
template <int kProduct, bool kPair>
__device__ __forceinline__ void linear_load_n(const LinearLoads& l, uint32_t dst, const void* tm,
                                              uint32_t full, int k, const LinearTile& t,
                                              const LinearParams& p) {
  for (int i = 0; i < l.b_boxes; ++i) {
    const uint32_t at = dst + kLinABytes + i * l.b_box_bytes;
    const int x = kProduct == LINEAR_GRAD_W ? l.n + 64 * i : k;
    const int y = kProduct == LINEAR_GRAD_W ? t.k_row + k : l.n + i * p.box_rows;
    if (kPair) tma_load_2d_pair(at, tm, full, x, y);
    else tma_load_2d(at, tm, full, x, y);
  }
}

// ------------------------------------------------------------------ epilogue
// 1 / (1 + e^-u) and 1 / (1 + e^u), with their relative accuracy on both sides: the
// exponential is at most 1, the denominator between 1 and 2.
struct Sigmoids {
  float up, down;
};
__device__ __forceinline__ Sigmoids sigmoids(float u) {
  const float e = __expf(-fabsf(u)), r = __fdividef(1.0f, 1.0f + e), s = e * r;
  return u < 0.0f ? Sigmoids{s, r} : Sigmoids{r, s};
}

// (1 + tanh u) / 2 is the sigmoid of 2u; 1.5957691 = 2 sqrt(2 / pi).
__device__ __forceinline__ float gelu_tanh_argument(float z) {
  return 1.5957691f * z * fmaf(0.044715f, z * z, 1.0f);
}

__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// P(Z <= z) of a standard normal Z.  Below 0
// it is e^(-z^2/2) f(|z|) with f(s) = erfcx(s / sqrt 2) / 2, here a polynomial in
// t = 1 / (1 + 0.3 s) that was fitted to f by weighted least squares (relative
// error 1.5e-7 for s up to 14, 4.7e-7 as evaluated in fp32; the whole has up to 2e-5
// at -13, by the exponential's argument): a subtraction from 1 would have no accuracy left there.
__device__ __forceinline__ float normal(float z) {
  const float s = fabsf(z), t = rcp_ftz(fmaf(0.3f, s, 1.0f));
  float f = 0.035674453f;
  f = fmaf(f, t, -0.15720180f);
  f = fmaf(f, t, 0.20635141f);
  f = fmaf(f, t, -0.053681802f);
  f = fmaf(f, t, 0.12856069f);
  f = fmaf(f, t, 0.099913761f);
  f = fmaf(f, t, 0.12075391f);
  f = fmaf(f, t, 0.11962930f);
  const float tail = __expf(-0.5f * z * z) * (f * t);
  return z < 0.0f ? tail : 1.0f - tail;
}

template <int kActivation>
__device__ __forceinline__ float activate(float z) {
  switch (kActivation) {
    case LINEAR_RELU: return z < 0.0f ? 0.0f : z;  // a NaN stays
    case LINEAR_GELU: return z * normal(z);
    case LINEAR_GELU_TANH: return z * sigmoids(gelu_tanh_argument(z)).up;
    case LINEAR_SILU: return z * sigmoids(z).up;
    default: return z;
  }
}

// z within -110 and 110, a NaN as it is.
__device__ __forceinline__ float within_110(float z) {
  float y;
  asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, 0fC2DC0000;\n\tmin.NaN.f32 %0, t, 0f42DC0000;\n\t}"
      : "=f"(y)
      : "f"(z));
  return y;
}

// act'(z).  Below 0, where it vanishes, it keeps its relative accuracy (but where it crosses zero):
// it is a product of an exponential, or a sigmoid, and a sum, and those carry a factor of 2^32 until
// the end, since the slope is up to 230 times the exponential and would be lost where that alone is
// below fp32's normal numbers (silu from -87.4 on, gelu from -13.2, gelu_tanh from -9.9).  Above 0 its
// accuracy is an absolute one; it is near 1 there.  Past 110 it is 0 or 1 in fp32, and products of
// what overflows and what vanishes there would be NaN.
template <int kActivation>
__device__ __forceinline__ float activation_slope(float z) {
  constexpr float kScale = 32.0f, kUnscale = 0x1p-32f;  // the factor, as an exponent, and its inverse
  if (kActivation == LINEAR_NONE) return 1.0f;
  if (kActivation == LINEAR_RELU) return z > 0.0f ? 1.0f : 0.0f;
  z = within_110(z);
  if (kActivation == LINEAR_GELU) {
    // as in `normal`, with a polynomial of degree 6: relative error 8.5e-6 (dz and bias of 8192 x
    // 4096 50 us with that of `normal`); act'(-|z|), of which act'(|z|) is the rest to 1
    const float s = fabsf(z), t = rcp_ftz(fmaf(0.3f, s, 1.0f));
    float f = -0.077096712f;
    f = fmaf(f, t, 0.21603487f);
    f = fmaf(f, t, -0.016945807f);
    f = fmaf(f, t, 0.14419527f);
    f = fmaf(f, t, 0.11374218f);
    f = fmaf(f, t, 0.12007421f);
    const float e = exp2_ftz(fmaf(s * s, -0.72134752f, kScale));
    const float low = e * (fmaf(s, -0.39894228f, f * t) * kUnscale);
    return z < 0.0f ? low : 1.0f - low;
  }
  // P (1 + z u' (1 - P)) with the sigmoid P of u(z); factors of -log2(e) in the exponent
  float exponent = fmaf(-1.4426950f, z, -kScale), zu = z;
  if (kActivation == LINEAR_GELU_TANH) {
    const float zz = z * z;
    exponent = fmaf(z, fmaf(-0.10294324f, zz, -2.3022082f), -kScale);
    zu = z * fmaf(0.21406445f, zz, 1.5957691f);
  }
  const float p = rcp_ftz(exp2_ftz(exponent) + kUnscale);  // 2^32 P
  return p * (fmaf(zu, fmaf(p, -kUnscale, 1.0f), 1.0f) * kUnscale);
}

// The activation of some values; the choice is made once for them.
template <int kN>
__device__ __forceinline__ void activate_all(float (&v)[kN], int activation) {
  const auto all = [&](auto a) {
#pragma unroll
    for (int e = 0; e < kN; ++e) v[e] = activate<decltype(a)::value>(v[e]);
  };
  switch (activation) {
    case LINEAR_RELU: return all(std::integral_constant<int, LINEAR_RELU>{});
    case LINEAR_GELU: return all(std::integral_constant<int, LINEAR_GELU>{});
    case LINEAR_GELU_TANH: return all(std::integral_constant<int, LINEAR_GELU_TANH>{});
    case LINEAR_SILU: return all(std::integral_constant<int, LINEAR_SILU>{});
  }
}

// 32 columns of a warp's 32 lanes of the accumulator, 32 rows of D's; zeros where nothing was summed
// (`any`).  The load and the wait for it are one statement: until the wait its registers
// are still being written, and the compiler, which does not know that, would move
// what it found in them, or use them for something else, in between.
__device__ __forceinline__ void linear_sums(uint32_t taddr, bool any, uint32_t (&r)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = any ? r[i] : 0u;
}

// 32 x 32 sums of a tile: lanes 32 q on of the accumulator, and columns 32 c on, `m` being
// the first of the M of the CTA.
struct LinearChunk {
  int64_t row;     // of D
  int32_t live;    // rows; none: not stored
  int32_t col;
};
template <int kProduct>
__device__ __forceinline__ LinearChunk linear_chunk(const LinearTile& t, int m, int q, int c,
                                                    const LinearParams& p) {
  LinearChunk o;
  o.row = (kProduct == LINEAR_GRAD_W ? static_cast<int64_t>(t.group) * p.m : 0) + t.n + 32 * c;
  o.live = min(32, t.n_count - 32 * c);
  o.col = m + 32 * q;
  if (o.col >= p.n) o.live = 0;
  return o;
}

// A chunk of D from the sums in registers, a column of it for each lane: each store of
// the warp is 64 neighbouring bytes of a row, whatever its alignment.  (Through shared
// memory, for 16 bytes a lane, the sums took as much of its bandwidth as the MMAs leave: grad_w of
// 4096 tokens x 8 of 64 experts 468 us, of which 104 were the epilogue's.)
template <typename T, int kProduct>
__device__ __forceinline__ void linear_store(float (&v)[32], const LinearParams& p, float bias,
                                             const T (&residual)[32], const LinearChunk& at,
                                             int lane) {
  if (at.col + lane >= p.n) return;
  const int64_t first = at.row * p.n + at.col + lane;
  const auto store = [&](uint16_t* to) {
    T* o = reinterpret_cast<T*>(to) + first;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i < at.live) *o = from_float<T>(v[i]);
      o += p.n;
    }
  };
  if (kProduct == LINEAR_FORWARD) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += bias;
    if (p.preact) store(p.preact);
    activate_all(v, p.activation);
    if (p.residual) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += to_float(residual[i]);
    }
  }
  store(p.out);
}

// kSplit: 32 x 32 sums in shared memory, rows of D of 128 bytes.  They go to another CTA's
// (a shared::cluster address) by whole rows: 16 bytes a lane, in 32 rows at once, took longer
// (128 x 512 x 2048 by eight CTAs, a tile of 256: 13.0 us, and 10.2 so).
__device__ __forceinline__ void linear_send(uint32_t buf, int lane, const uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(buf + 128u * i + 4u * lane), "r"(r[i])
                 : "memory");
}

// The sums of `parts` buffers `part_bytes` apart, added in order.
__device__ __forceinline__ void linear_add_parts(uint32_t buf, int parts, uint32_t part_bytes,
                                                 int lane, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
#pragma unroll 1
  for (int s = 0; s < parts; ++s) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float part;
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(part)
                   : "r"(buf + s * part_bytes + 128u * i + 4u * lane)
                   : "memory");
      v[i] += part;
    }
  }
}

// ------------------------------------------------------------------ grad_bias
// The sums of dz over strips of strip_rows rows (the last of a group is shorter) are
// rows of `strips`, those of group g from offsets[g] / strip_rows + g on: no group
// needs to know how many strips others have.
__host__ __device__ __forceinline__ int strip_of(int row, int group, int strip_rows) {
  return row / strip_rows + group;
}

// Floats between the strips.
__host__ __device__ constexpr int64_t strip_ld(int64_t n) { return (n + 3) & ~int64_t{3}; }

// grad_bias from the strips, by warps first, first + step ... of the grid; in the products'
// kernels by the epilogue's, which wait for the first sums anyway.  A warp has 32 columns of a
// group at a time: a quarter of its lanes takes every fourth strip, with eight of them asked for
// at once, and the four sums are added at the end, always in the same order.  (A column for each
// thread, one strip after the other, took 16 us for the 128 strips of 8192 rows.)
template <typename T>
__device__ __forceinline__ void linear_sum_strips(const LinearParams& p, const GroupStart* start,
                                                  int64_t first, int64_t step, int lane) {
  constexpr int kAhead = 8;
  const int per = (p.m + 31) >> 5;
  const int64_t units = static_cast<int64_t>(p.groups) * per;
  const int64_t ld = strip_ld(p.m);
  for (int64_t u = first; u < units; u += step) {
    const int g = static_cast<int>(u / per);
    const int c = static_cast<int>(u - static_cast<int64_t>(g) * per) * 32 + 4 * (lane & 7);
    const int row = start[g].row;
    const int count = (start[g + 1].row - row + p.strip_rows - 1) / p.strip_rows;
    const float* const at = p.strips + strip_of(row, g, p.strip_rows) * ld + min(c, (p.m - 1) & ~3);
    float sum[4] = {};
    for (int s0 = lane >> 3; s0 < count; s0 += 4 * kAhead) {
      float4 v[kAhead];  // past the last: the last again (a load that depends is not sent ahead)
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        v[e] = __ldcg(reinterpret_cast<const float4*>(at + min(s0 + 4 * e, count - 1) * ld));
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const bool live = s0 + 4 * e < count;
        sum[0] += live ? v[e].x : 0.0f;
        sum[1] += live ? v[e].y : 0.0f;
        sum[2] += live ? v[e].z : 0.0f;
        sum[3] += live ? v[e].w : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 8);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 16);
    }
    if (lane < 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < p.m)
          reinterpret_cast<T*>(p.grad_bias)[static_cast<int64_t>(g) * p.m + c + i] =
              from_float<T>(sum[i]);
    }
  }
}

template <typename T>
__device__ __forceinline__ void linear_sum_strips(const LinearParams& p, const GroupStart* start) {
  if (!p.strips) return;
  // the CTAs' first epilogue warps before their second ones
  linear_sum_strips<T>(p, start,
                       static_cast<int64_t>(threadIdx.x / 32 - 2) * gridDim.x + blockIdx.x,
                       static_cast<int64_t>(gridDim.x) * kLinEpiWarps, threadIdx.x & 31);
}

// What a lane's column of D has added to it.
template <typename T, int kProduct>
__device__ __forceinline__ float linear_bias(const LinearParams& p, int group, int col) {
  if (kProduct != LINEAR_FORWARD || !p.bias || col >= p.n) return 0.0f;
  return to_float(reinterpret_cast<const T*>(p.bias)[static_cast<int64_t>(group) * p.n + col]);
}
template <typename T, int kProduct>
__device__ __forceinline__ void linear_residual(T (&residual)[32], const LinearParams& p,
                                                const LinearChunk& at, int lane) {
  const int col = at.col + lane;
  if (kProduct != LINEAR_FORWARD || !p.residual || col >= p.n) return;
  const T* from = reinterpret_cast<const T*>(p.residual) + at.row * p.ldr + col;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (i < at.live) residual[i] = *from;
    from += p.ldr;
  }
}

// An epilogue warp's chunks of a tile: those of lane quadrant q, columns 32 half, 32 (half + 2)
// ...  `wait` waits for the accumulator and `release` gives it back, by one lane, once
// the warp's last chunk of it is in registers.  False: the wait gave up.
template <typename T, int kProduct, typename Wait, typename Release>
__device__ __forceinline__ bool linear_epilogue(const LinearTile& tile, int m, int q, int half,
                                                uint32_t t_row, const LinearParams& p, int lane,
                                                Wait wait, Release release) {
  const auto let_go = [&] {
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) release();
  };
  const int chunks = m + 32 * q < p.n ? (tile.n_count + 31) >> 5 : 0;
  const float bias = linear_bias<T, kProduct>(p, tile.group, m + 32 * q + lane);
  if (!wait()) return false;
  tc_fence_after_sync();
  if (chunks <= half) let_go();
  for (int c = half; c < chunks; c += 2) {
    const LinearChunk at = linear_chunk<kProduct>(tile, m, q, c, p);
    T residual[32];
    linear_residual<T, kProduct>(residual, p, at, lane);
    uint32_t r[32];
    linear_sums(t_row + 32 * c, tile.k_len > 0, r);
    if (c + 2 >= chunks) let_go();
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
    linear_store<T, kProduct>(v, p, bias, residual, at, lane);
  }
  return true;
}

// Rows of no group are zero, by every epilogue thread of the grid.
template <int kProduct>
__device__ __forceinline__ void linear_zero_tail(const LinearParams& p, const GroupStart* start) {
  if (kProduct == LINEAR_GRAD_W || !p.offsets) return;
  const int64_t from = static_cast<int64_t>(start[p.groups].row) * p.n;
  const int64_t end = static_cast<int64_t>(p.rows) * p.n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (32 * kLinEpiWarps);
  for (int64_t i = from + static_cast<int64_t>(blockIdx.x) * (32 * kLinEpiWarps) + threadIdx.x - 64;
       i < end; i += step) {
    p.out[i] = 0;
    if (kProduct == LINEAR_FORWARD && p.preact) p.preact[i] = 0;
  }
}

}  // namespace gb300
