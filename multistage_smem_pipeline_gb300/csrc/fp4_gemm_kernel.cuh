// The 4-bit product on the tensor cores.
//
// D[r][n] = alpha sum_k a[r][k] b[g][n][k] for the rows r of group g.  The
// weights are the instruction's M operand (128 rows a tile) and the
// activations its N operand (1 to 128 rows a tile here, to 256 in the kernel
// over CTA pairs): N may be any multiple of 16, so that an expert with few rows
// costs few columns.  A tile's accumulator is then D transposed: lane = output
// n, column = row r.
//
// With few rows what bounds it are the weights' bytes from memory: 1 x 155648 x
// 4096 nvfp4 takes 55 us (6.5 TB/s), 1 x 14336 x 4096 7.3 (4.5 TB/s, of which
// 2.5 us are a launch's beginning and end), 8 tokens over 64 experts (32 of
// them at most, 2048 x 4096 each) 19.5.  With many rows and a short k it is the
// stores, two bytes a lane: 8192 x 4096 x 256 in 16 us.  Staged through shared
// memory for 16 bytes a lane, with the barriers between warps that takes, they
// were slower (128 x 14336 x 4096 8.7 us against 8.2, and twice as long where
// D's rows are not aligned).
//
// Inside a CTA, one per SM, each walking the list of tiles:
//   warps 0 and 10 -- producers, of the weights and of the rows: per 256 columns
//       of k (128 bytes of codes a row), TMA boxes of codes and a bulk copy of
//       the scale chunks into a ring of stages;
//   warp 1 -- copies the stage's scales into tensor memory
//       (tcgen05.cp, 512 bytes = 128 rows x 4 blocks at a time, replicated to
//       the four lane quadrants) and issues a block-scaled MMA per 64 columns;
//   warps 2 .. 9 -- epilogue: four warps, one per lane quadrant, for each of the
//       two accumulators; they take a tile to registers, round it, let the
//       accumulator go, and store.
// Every ring slot has its own columns of tensor memory for scales: a slot's
// copies begin after its full barrier, hence after its empty one, which the
// commit of the MMAs that read those columns completed.
//
// Waits are bounded as in the fp16 kernels: on expiry the error word is set,
// all roles leave their loops, what is in flight is drained, and tensor
// memory is freed.
#pragma once
#include <cuda.h>

#include "fp4.cuh"

namespace gb300 {

constexpr int kGemmM = 128;           // weight rows per tile
constexpr int kGemmBytesK = 128;      // codes of a row per stage: 256 elements
constexpr int kGemmEpiWarps = 8;
constexpr int kGemmRowWarp = 2 + kGemmEpiWarps;  // the second producer
constexpr int kGemmThreads = 96 + 32 * kGemmEpiWarps;
constexpr int kGemmMaxStages = 8;
constexpr uint32_t kWBytes = kGemmM * kGemmBytesK;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemScales = 256;  // first column of the scales
constexpr int kErrorWords = 64;
constexpr uint32_t kGemmSmemLimit = 232448;

enum GemmWait : uint32_t { kWaitEmpty = 1, kWaitFull = 2, kWaitTmemEmpty = 3, kWaitTmemFull = 4,
                          kWaitParts = 5 };

struct Fp4GemmParams {
  const uint8_t* w_scales;
  const uint8_t* x_scales;
  int64_t w_tile_bytes, x_tile_bytes;
  uint16_t* d;
  const int32_t* offsets;  // of the rows' groups; null: uniform groups
  int64_t rows, group_rows, n_out;
  int32_t groups, num_kb;
  int32_t m_tiles;         // weight tiles (of the kernel's height) per group
  int32_t w_group_tiles;   // scale tiles of the weights per group
  int32_t tile_chunks;     // chunks of a scale tile
  int32_t box_rows;        // activation rows per TMA box
  int32_t stages;
  int32_t split;           // CTAs that share a tile's k; 1: none do
  float pre, alpha;        // the sums' factor, in two where fp32 has no normal number for it
  uint64_t timeout_ns;
  int32_t inject;          // 1: leave out each CTA's first loads
  int32_t error_word;      // where this call's errors go
};

constexpr int kGemmBN = 128;  // activation rows per tile, at most

template <int kFormat>
struct Fp4GemmShape {
  static constexpr uint32_t kScaleStage = chunks_per_stage(kFormat) * kChunkBytes;
  static constexpr uint32_t kXBytes = kGemmBN * kGemmBytesK;
  static constexpr uint32_t kStageBytes = kWBytes + kXBytes + 2 * kScaleStage;
  // columns of scales per slot: 4 per chunk and 128 rows
  static constexpr uint32_t kWCols = 4 * chunks_per_stage(kFormat);
  static constexpr uint32_t kSlotCols = 2 * kWCols;
  static constexpr int kSlots = (kTmemCols - kTmemScales) / kSlotCols;
  static int stages_that_fit(uint32_t fixed) {
    return std::min<int>({static_cast<int>((kGemmSmemLimit - fixed) / kStageBytes), kSlots,
                          kGemmMaxStages});
  }
};

// A split tile's partial sums: 128 outputs x 128 rows in fp32.
constexpr uint32_t kSplitBytes = kGemmM * kGemmBN * 4;

// Shared memory past the ring (and the partial sums): barriers, then the tensor memory address, the
// abort flag, and where each group starts.
constexpr uint32_t kGemmBars = 2 * kGemmMaxStages + 6;
__host__ __device__ constexpr uint32_t gemm_fixed_bytes(int groups) {
  return 8 * kGemmBars + 16 + 8 * (groups + 1) + 1024;  // 1 KiB to align the ring
}

// ------------------------------------------------------------------ PTX
// Instruction descriptor of the block-scaled kinds: A and B E2M1 (bits 7-9
// and 10-11 = 1), both K-major, N >> 3 in bits 17-22, the scales' type in bit
// 23 (0: E4M3, 1: E8M0), M >> 4 in bits 24-28; bits 4-5 and 29-30 say which
// bytes of a 32-bit column hold the scales of B and A.
template <int kFormat>
__host__ __device__ constexpr uint32_t fp4_idesc(int m, int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (kFormat == FP4_MX ? 1u << 23 : 0u) | (static_cast<uint32_t>(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t fp4_idesc_scale_bytes(int first) {
  return (static_cast<uint32_t>(first) << 4) | (static_cast<uint32_t>(first) << 29);
}

template <int kFormat>
__device__ __forceinline__ void umma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t a_scales, uint32_t b_scales,
                                         uint32_t accumulate) {
  if (kFormat == FP4_NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
        : "memory");
}

// 32 rows x 16 bytes of shared memory to 32 lanes x 4 columns, in all four
// lane quadrants.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// Shared-memory descriptor of an unswizzled run of 16-byte rows: 8-row groups
// 128 bytes apart (stride byte offset), descriptor version 1.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// ------------------------------------------------------------------ waits
// The first error of the launches on a given stream (the host maps streams to
// words); 0: none.
__device__ uint32_t g_fp4_error[kErrorWords];

__device__ __forceinline__ void record_timeout(volatile int* abort_flag, uint32_t site,
                                               const Fp4GemmParams& p) {
  *abort_flag = 1;
  atomicCAS(&g_fp4_error[p.error_word], 0u,
            static_cast<uint32_t>(GEMM_ERR_TIMEOUT) | (site << 8));
}

__device__ __forceinline__ bool gemm_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint32_t site, const Fp4GemmParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > p.timeout_ns) {
        record_timeout(abort_flag, site, p);
        return false;
      }
    }
  }
}

// A wait for data from other CTAs of the cluster.
__device__ __forceinline__ bool gemm_wait_cluster(uint32_t bar, uint32_t parity,
                                                  volatile int* abort_flag, uint32_t site,
                                                  const Fp4GemmParams& p) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 31u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > p.timeout_ns) {
        record_timeout(abort_flag, site, p);
        return false;
      }
    }
  }
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// The same wait by a whole warp: it goes on, or gives up, together.
__device__ __forceinline__ bool gemm_wait_warp(uint32_t bar, uint32_t parity,
                                               volatile int* abort_flag, uint32_t site,
                                               const Fp4GemmParams& p) {
  return __all_sync(0xffffffffu, gemm_wait(bar, parity, abort_flag, site, p));
}

__device__ __forceinline__ void gemm_wait_drain(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return;
    if ((it & 31u) == 0 && global_timer_ns() - t0 > timeout_ns) return;
  }
}

// ------------------------------------------------------------------ tiles
struct GemmTile {
  int32_t x_row;    // first row of the activations (and of D)
  int32_t x_tile;   // its scale tile
  int32_t count;    // rows
  int32_t group, m; // weight tile m of the group
};

// A group by offsets, in shared memory: every role looks each tile's group up
// (from global memory: 129.0 us for 4096 tokens x 8 of 64 experts, against 128.2).
struct GroupStart {
  int32_t tiles;  // row tiles of the groups before it
  int32_t row;    // its first row
};

// Tile t: groups in order; in a group, kRaster row tiles at a time walk over the
// weight tiles together, so that what runs at once shares operands in L2.  (The
// host keeps the number of tiles within 32 bits: every role works this out for
// every tile, and with short k loops it shows.)
constexpr int kRaster = 8;

template <int kBN>
__device__ __forceinline__ GemmTile gemm_tile(int t, const Fp4GemmParams& p, const GroupStart* start) {
  GemmTile o;
  int first, rows;
  if (p.offsets) {
    int lo = 0, hi = p.groups - 1;  // the last group with tiles * m_tiles <= t before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid].tiles * p.m_tiles <= t) lo = mid;
      else hi = mid - 1;
    }
    o.group = lo;
    t -= start[lo].tiles * p.m_tiles;
    first = start[lo].row;
    rows = start[lo + 1].row - first;
    o.x_tile = first / kTileRows + lo;
  } else {
    rows = static_cast<int>(p.group_rows);
    o.group = 0;
    if (p.groups > 1) {
      const int per = (rows + kBN - 1) / kBN * p.m_tiles;
      o.group = t / per;
      t -= o.group * per;
    }
    first = o.group * rows;
    o.x_tile = o.group * ((rows + kTileRows - 1) / kTileRows);
  }
  int xt;
  if (rows <= kBN) {
    xt = 0;
    o.m = t;
  } else {
    const int x_tiles = (rows + kBN - 1) / kBN;
    const int band = t / (kRaster * p.m_tiles);
    const int in = t - band * kRaster * p.m_tiles;
    const int wide = min(kRaster, x_tiles - band * kRaster);
    if (wide == kRaster) {
      xt = in % kRaster;
      o.m = in / kRaster;
    } else {
      o.m = in / wide;
      xt = in - o.m * wide;
    }
    xt += band * kRaster;
  }
  o.x_row = first + xt * kBN;
  o.x_tile += xt * (kBN / kTileRows);
  o.count = min(kBN, rows - xt * kBN);
  return o;
}

template <typename T>
__device__ __forceinline__ uint32_t pack_two(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack_two<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack_two<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------------------ epilogue
// One warp's part of a tile's accumulator, lanes 32 q .. 32 q + 31 and four
// 32-column chunks (first, first + kStep ...): to registers in one go, rounded in place (element i
// of a chunk's array then holds columns 2i and 2i + 1), the accumulator let go
// by `release`, and stored; a lane is an output n, so a store of the warp
// writes 32 neighbouring outputs of one row.
template <typename T, int kStep, typename Release>
__device__ __forceinline__ void store_tile(uint32_t t_row, int first, int count,
                                           const Fp4GemmParams& p, uint16_t* d, bool live,
                                           Release release) {
  constexpr int kMine = 4;
  uint32_t r[kMine][32];
#pragma unroll
  for (int c = 0; c < kMine; ++c)
    if (32 * (kStep * c + first) < count)
      tmem_ld_32x32b_x32(t_row + 32 * (kStep * c + first), r[c]);
  tmem_ld_wait();
  release();
  if (p.pre != 1.0f) {
#pragma unroll
    for (int c = 0; c < kMine; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) r[c][i] = __float_as_uint(p.pre * __uint_as_float(r[c][i]));
  }
#pragma unroll
  for (int c = 0; c < kMine; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      r[c][i] = pack_two<T>(p.alpha * __uint_as_float(r[c][2 * i]),
                            p.alpha * __uint_as_float(r[c][2 * i + 1]));
  if (!live) return;
#pragma unroll
  for (int c = 0; c < kMine; ++c) {
    const int col = 32 * (kStep * c + first);
    if (col >= count) break;
    uint16_t* to = d + col * p.n_out;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (col + i < count) *to = static_cast<uint16_t>(r[c][i >> 1] >> (16 * (i & 1)));
      to += p.n_out;
    }
  }
}

// A CTA's part of a split tile: thread `out` of 128 (its output) and the 32-column
// chunks of its warp.  Slot s of `partial` holds part s's sums for this CTA's
// columns: [s][chunk][output][32 / split].
template <typename T>
__device__ __forceinline__ void store_split_tile(uint32_t t_row, int out, int half, int count,
                                                 int part, const Fp4GemmParams& p, uint32_t partial,
                                                 uint32_t parts_bar, volatile int* abort_flag,
                                                 uint16_t* d, bool live) {
  const int quads = 8 / p.split;  // groups of four columns a CTA has of a chunk
  const auto slot = [&](int s, int chunk) {
    return partial + static_cast<uint32_t>(((s * 4 + chunk) * kGemmM + out) * quads) * 16u;
  };
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int chunk = 2 * c + half;
    if (32 * chunk >= count) break;
    uint32_t r[32];
    tmem_ld_32x32b_x32(t_row + 32 * chunk, r);
    tmem_ld_wait();
    const uint32_t mine = slot(part, chunk);
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const int to = g / quads;
      const uint32_t at = mine + (g - to * quads) * 16u;
      if (to == part)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[4 * g]),
                     "r"(r[4 * g + 1]), "r"(r[4 * g + 2]), "r"(r[4 * g + 3])
                     : "memory");
      else
        st_async_cluster_v4(mapa_shared(at, to), r[4 * g], r[4 * g + 1], r[4 * g + 2],
                            r[4 * g + 3], mapa_shared(parts_bar, to));
    }
  }
  if (!gemm_wait_cluster(parts_bar, 0, abort_flag, kWaitParts, p)) return;
  if (!live) return;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int chunk = 2 * c + half;
    for (int g = 0; g < quads; ++g) {
      const int col = 32 * chunk + 4 * (part * quads + g);
      if (col >= count) break;
      float sum[4] = {};
      for (int s = 0; s < p.split; ++s) {
        float v[4];
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "r"(slot(s, chunk) + g * 16u)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += v[i];
      }
      if (p.pre != 1.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] *= p.pre;
      }
      const uint32_t w[2] = {pack_two<T>(p.alpha * sum[0], p.alpha * sum[1]),
                             pack_two<T>(p.alpha * sum[2], p.alpha * sum[3])};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < count)
          d[(col + i) * p.n_out] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// Rows of no group are zero: elements [from, end) of D, by every epilogue
// thread of the grid.
__device__ __forceinline__ void zero_tail(const Fp4GemmParams& p, const GroupStart* start) {
  if (!p.offsets) return;
  const int64_t from = static_cast<int64_t>(start[p.groups].row) * p.n_out;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (32 * kGemmEpiWarps);
  for (int64_t i = from + static_cast<int64_t>(blockIdx.x) * (32 * kGemmEpiWarps) + threadIdx.x - 64;
       i < p.rows * p.n_out; i += step)
    p.d[i] = 0;
}

// Where each group starts, and the end, by one warp.  All offsets of 128 groups
// are asked for at once: nothing can be loaded before this is done, and one
// latency of memory is 0.4 us.
template <int kBN>
__device__ __forceinline__ void find_groups(const Fp4GemmParams& p, GroupStart* start, int lane) {
  constexpr int kAhead = 4;
  int32_t total = 0;
  for (int g0 = 0; g0 <= p.groups; g0 += 32 * kAhead) {
    int32_t row[kAhead + 1];
#pragma unroll
    for (int i = 0; i <= kAhead; ++i) row[i] = p.offsets[min(g0 + 32 * i + lane, p.groups)];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int g = g0 + 32 * i + lane;
      const int32_t next = __shfl_down_sync(0xffffffffu, row[i], 1);
      const int32_t first = __shfl_sync(0xffffffffu, row[i + 1], 0);
      const int32_t n = ((lane < 31 ? next : first) - row[i] + kBN - 1) / kBN;  // 0 past the last
      int32_t upto = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
      }
      if (g <= p.groups) start[g] = GroupStart{total + upto - n, row[i]};
      total += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
}

// ------------------------------------------------------------------ kernel
// kSplit: few tiles.  A cluster of p.split CTAs (2, 4 or 8) shares one tile, each
// taking its part of k; then every CTA sends each other one its partial sums
// for that one's 32 / split columns of each chunk of 32, straight from
// registers into its shared memory, and adds up what it receives for its own
// in the order of the parts.  No sum depends on who came first.  The grid has a
// cluster for every tile there may be.
template <typename T, int kFormat, bool kSplit>
__global__ void __launch_bounds__(kGemmThreads, 1)
    fp4_gemm_tc(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const Fp4GemmParams p) {
  constexpr int kBN = kGemmBN;
  static_assert(kBN == kTileRows, "a row tile is a scale tile");
  using S = Fp4GemmShape<kFormat>;
  constexpr int kChunks = chunks_per_stage(kFormat);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.stages;
  const uint32_t partial = base + stages * S::kStageBytes;
  const uint32_t bars = partial + (kSplit ? kSplitBytes : 0u);
  const int part = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
  const int first_tile = kSplit ? blockIdx.x / p.split : blockIdx.x;
  const int tile_step = kSplit ? INT_MAX / 4 : gridDim.x;  // kSplit: one tile
  const int kb_first = kSplit ? part * p.num_kb / p.split : 0;
  const int kb_end = kSplit ? (part + 1) * p.num_kb / p.split : p.num_kb;
  const auto full_bar = [&](int s) { return bars + 8u * s; };
  const auto empty_bar = [&](int s) { return bars + 8u * (kGemmMaxStages + s); };
  const auto tfull_bar = [&](int b) { return bars + 8u * (2 * kGemmMaxStages + b); };
  const auto tempty_bar = [&](int b) { return bars + 8u * (2 * kGemmMaxStages + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * kGemmMaxStages + 4);
  const uint32_t parts_bar = drain_bar + 8;  // the other parts' sums have come
  uint8_t* const misc = smem + (bars - base) + 8 * kGemmBars;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  GroupStart* const start = reinterpret_cast<GroupStart*>(misc + 16);

  if (threadIdx.x == 0) {
    grid_launch_dependents();
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), kGemmEpiWarps / 2);
    }
    mbar_init(drain_bar, 1);
    mbar_init(parts_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  if (p.offsets && warp == 2) find_groups<kBN>(p, start, lane);
  tc_fence_before_sync();
  if (kSplit) cluster_sync();  // the others' barriers exist
  else __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int tiles =
      (p.offsets ? start[p.groups].tiles
                 : p.groups * ((static_cast<int>(p.group_rows) + kBN - 1) / kBN)) * p.m_tiles;

  if (warp == 0 || warp == kGemmRowWarp) {
    // ---------------------------------------------------------- producers
    // Warp 0 loads the weights and their scales, the other the rows and theirs:
    // what a copy costs its issuer bounds one warp alone.
    // The whole warp runs the loop and one lane issues: the values that the
    // copies take are then the same in every lane, which costs the issue of a
    // copy far less than a loop inside one lane's branch does.
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int t = first_tile; ok && t < tiles; t += tile_step) {
      const GemmTile tile = gemm_tile<kBN>(t, p, start);
      const int boxes = (tile.count + p.box_rows - 1) / p.box_rows;
      const uint32_t bytes = kWBytes + static_cast<uint32_t>(boxes * p.box_rows) * kGemmBytesK +
                             2 * S::kScaleStage;
      const int w_row = static_cast<int>(tile.group * p.n_out + tile.m * kGemmM);
      const int x_row = tile.x_row;
      const uint8_t* w_scales =
          p.w_scales +
          (static_cast<int64_t>(tile.group) * p.w_group_tiles + tile.m) * p.w_tile_bytes +
          static_cast<int64_t>(kb_first) * S::kScaleStage;
      const uint8_t* x_scales = p.x_scales + tile.x_tile * p.x_tile_bytes +
                                static_cast<int64_t>(kb_first) * S::kScaleStage;
      for (int kb = kb_first; kb < kb_end; ++kb) {
        if (!gemm_wait_warp(empty_bar(stage), phase ^ 1u, abort_flag, kWaitEmpty, p)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t w_dst = base + stage * S::kStageBytes;
          const uint32_t x_dst = w_dst + kWBytes;
          const uint32_t s_dst = x_dst + S::kXBytes;
          const uint32_t full = full_bar(stage);
          if (warp == 0) {
            mbar_arrive_expect_tx(full, bytes);
            if (!(p.inject && issued == 0))
              tma_load_2d(w_dst, &tmW, full, kb * kGemmBytesK, w_row);
            bulk_load(s_dst, w_scales, S::kScaleStage, full);
          } else {
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(x_dst + b * p.box_rows * kGemmBytesK, &tmX, full, kb * kGemmBytesK,
                          x_row + b * p.box_rows);
            bulk_load(s_dst + S::kScaleStage, x_scales, S::kScaleStage, full);
          }
        }
        __syncwarp();
        w_scales += S::kScaleStage;
        x_scales += S::kScaleStage;
        ++issued;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // every load has landed before the CTA may end
    const uint32_t first = issued > static_cast<uint32_t>(stages) ? issued - stages : 0u;
    for (uint32_t i = first; i < issued; ++i)
      gemm_wait_drain(full_bar(i % stages), (i / stages) & 1u, p.timeout_ns);
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // As the producer: the warp loops, one lane issues, and the descriptors
    // are one addition away from those of stage 0.  Measured at 8192^3: 538 us
    // with one lane's loop and descriptors made on the spot, 345 with these
    // descriptors, 268 with the warp's loop as well.
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    const uint64_t w_desc0 = sw128_kmajor_desc(base);
    const uint64_t s_desc0 = scale_desc(base + kWBytes + S::kXBytes);
    for (int t = first_tile; ok && t < tiles; t += tile_step) {
      const GemmTile tile = gemm_tile<kBN>(t, p, start);
      const uint32_t idesc = fp4_idesc<kFormat>(kGemmM, (tile.count + 15) & ~15);
      if (!gemm_wait_warp(tempty_bar(acc), acc_phase ^ 1u, abort_flag, kWaitTmemEmpty, p)) break;
      tc_fence_after_sync();
      const uint32_t d_tmem = tmem + static_cast<uint32_t>(acc * kBN);
      for (int kb = kb_first; kb < kb_end; ++kb) {
        if (!gemm_wait_warp(full_bar(stage), phase, abort_flag, kWaitFull, p)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (elect_one()) {
          const uint64_t at = static_cast<uint64_t>((stage * S::kStageBytes) >> 4);
          const uint64_t s_desc = s_desc0 + at;
          const uint32_t w_cols = tmem + kTmemScales + stage * S::kSlotCols;
          const uint32_t x_cols = w_cols + S::kWCols;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            tmem_copy_scales(w_cols + 4 * c, s_desc + ((c * kChunkBytes) >> 4));
            tmem_copy_scales(x_cols + 4 * c, s_desc + ((S::kScaleStage + c * kChunkBytes) >> 4));
          }
          const uint64_t w_desc = w_desc0 + at;
          const uint64_t x_desc = w_desc + (kWBytes >> 4);
#pragma unroll
          for (int s = 0; s < 4; ++s) {  // 64 columns each; past k codes and scales are zero
            const int chunk = kFormat == FP4_NV ? s : s >> 1;
            const int byte = kFormat == FP4_NV ? 0 : (s & 1) * 2;
            umma_fp4<kFormat>(d_tmem, w_desc + 2u * s, x_desc + 2u * s,
                              idesc | fp4_idesc_scale_bytes(byte), w_cols + 4 * chunk,
                              x_cols + 4 * chunk, kb != kb_first || s != 0);
          }
          umma_commit(empty_bar(stage));
        }
        __syncwarp();
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elect_one()) umma_commit(tfull_bar(acc));
      __syncwarp();
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (elect_one()) umma_commit(drain_bar);
    __syncwarp();
    gemm_wait_drain(drain_bar, 0, p.timeout_ns);
  } else {
    // ---------------------------------------------------------- epilogue
    // Two groups of four warps, one per accumulator: while one stores a tile the
    // other reads the next.  (A split tile is shared by both, by chunks.)
    const int q = warp & 3;               // the lane quadrant this warp may read
    const int group = (warp - 2) >> 2;
    uint32_t acc_phase = 0;
    for (int t = first_tile + (kSplit ? 0 : group * tile_step); t < tiles;
         t += (kSplit ? 1 : 2) * tile_step) {
      const GemmTile tile = gemm_tile<kBN>(t, p, start);
      const int acc = kSplit ? 0 : group;
      int ok = 0;
      if (lane == 0) ok = gemm_wait(tfull_bar(acc), acc_phase, abort_flag, kWaitTmemFull, p);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(acc * kBN);
      const int64_t n = static_cast<int64_t>(tile.m) * kGemmM + q * 32 + lane;
      uint16_t* const d = p.d + tile.x_row * p.n_out + n;
      if (kSplit) {
        if (warp == 2 && lane == 0)  // 128 outputs x 32 / split columns of each chunk, from each
          mbar_arrive_expect_tx(parts_bar, (p.split - 1) * ((tile.count + 31) / 32) *
                                               (kGemmM * 128 / p.split));
        store_split_tile<T>(t_row, q * 32 + lane, group, tile.count, part, p, partial, parts_bar,
                            abort_flag, d, n < p.n_out);
        continue;
      }
      store_tile<T, 1>(t_row, 0, tile.count, p, d, n < p.n_out, [&] {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
      });
      acc_phase ^= 1u;
    }
    zero_tail(p, start);
  }
  __syncwarp();
  tc_fence_before_sync();
  if (kSplit) cluster_sync();  // no CTA's shared memory goes while another may write to it
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace gb300
