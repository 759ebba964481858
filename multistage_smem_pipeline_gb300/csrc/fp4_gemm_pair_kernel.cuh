// The 4-bit product over CTA pairs (tcgen05 cta_group::2).
//
// A pair owns 256 outputs x up to 256 rows.  Each CTA loads its own 128 rows of
// weights, its half of the activations' rows, the scales of its weights and one
// of the two tiles of the activations' scales, which goes to both; the even CTA
// issues, and each CTA accumulates its 128 outputs in its own tensor memory.
//
// What bounds it is how operands get to the MMAs: per 256 columns of k an SM takes
// in 38 KiB and its MMAs read 32 KiB of codes and 6 KiB of scales in 512 cycles,
// together more than shared memory's 128 bytes a cycle; a single CTA's 128 x 256
// tile would take in 54 and read 54.  At 8192^3 the loads alone take 124 us (65
// bytes a cycle into each SM, which looks like what comes in from L2), the MMAs alone 136 (of
// which 14 are the accumulator changing hands, as there is no room for two of
// 256 columns and the scales), both 151, and the stores make it 164
// (6.7 PFLOP/s).  Codes and scales have rings of their own because tensor memory
// has room for five blocks' nvfp4 scales and shared memory for six of codes: with
// 3, 4, 5 and 6 blocks of codes 8192^3 takes 208, 177, 165 and 164 us, and 4096
// tokens x 8 of 64 experts, 4096 -> 2048, 153, 134, 129 and 125.
// Tried and no faster: 384 rows a tile (176 us: 10 waves where 9.3 would do), two
// pairs sharing the rows by multicast (177: 36 such clusters fit where 38 would
// fill the SMs), L2 prefetch of the weights (194).  With ragged groups, tiles
// handed out as pairs get free (clusters not yet begun taken over): 131 us for the
// 4096 tokens where the fixed stride took 128, though the stride leaves the last
// pair 13 % more work than the mean; pairs that run in step share operands in L2.
//
// Barriers as in the fp16 pair kernel: `full` in the even CTA counts both
// CTAs' bytes; `empty` and `tfull` are in both, committed to both; `tempty` in
// the even CTA takes every epilogue warp of both.
#pragma once
#include "fp4_gemm_kernel.cuh"

namespace gb300 {

template <int kFormat>
struct Fp4PairShape {
  static constexpr int kBN = 256;
  static constexpr int kXTiles = 2;
  static constexpr uint32_t kScaleStage = chunks_per_stage(kFormat) * kChunkBytes;
  static constexpr uint32_t kXBytes = kBN / 2 * kGemmBytesK;
  static constexpr uint32_t kStageBytes = kWBytes + kXBytes;  // codes
  static constexpr uint32_t kSlotBytes = kScaleStage * (1 + kXTiles);
  static constexpr uint32_t kWCols = 4 * chunks_per_stage(kFormat);
  static constexpr uint32_t kSlotCols = kWCols * (1 + kXTiles);
  static constexpr int kSlots = (kTmemCols - kTmemScales) / kSlotCols;
  static __host__ __device__ int slots(int stages) { return stages < kSlots ? stages : kSlots; }
  static uint32_t ring_bytes(int stages) { return stages * kStageBytes + slots(stages) * kSlotBytes; }
  static int stages_that_fit(uint32_t fixed) {
    int s = kGemmMaxStages;
    while (ring_bytes(s) + fixed > kGemmSmemLimit) --s;
    return s;
  }
};

template <int kFormat>
__device__ __forceinline__ void umma_fp4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t a_scales, uint32_t b_scales,
                                              uint32_t accumulate) {
  if (kFormat == FP4_NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
        : "memory");
}

// One box into the shared memory of every CTA of `cta_mask`, at the same
// offset; its bytes complete on the barrier at `bar`'s offset in the even CTA of
// each of those CTAs' pairs (`bar`: the address in this CTA's).
__device__ __forceinline__ void tma_load_2d_pair_mc(uint32_t dst, const void* tmap, uint32_t bar,
                                                    int32_t x, int32_t y, uint16_t cta_mask) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".multicast::cluster [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "h"(cta_mask)
      : "memory");
}

// In each CTA of the pair, from its own shared memory to its own tensor memory.
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// tmSW, tmSX: the scales as rows of one chunk (128 words).
template <typename T, int kFormat>
__global__ void __launch_bounds__(kGemmThreads, 1)
    fp4_gemm_pair(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ CUtensorMap tmSW,
                  const __grid_constant__ CUtensorMap tmSX, const Fp4GemmParams p) {
  using S = Fp4PairShape<kFormat>;
  constexpr int kBN = S::kBN;
  static_assert(kBN == 1 << 8, "find_groups below");
  constexpr int kChunks = chunks_per_stage(kFormat);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.stages, slots = S::slots(stages);
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  constexpr uint16_t kBoth = 0x3;
  const uint32_t scales = base + stages * S::kStageBytes;
  const uint32_t bars = scales + slots * S::kSlotBytes;
  const auto full_bar = [&](int s) { return bars + 8u * s; };
  const auto empty_bar = [&](int s) { return bars + 8u * (kGemmMaxStages + s); };
  const uint32_t tfull_bar = bars + 8u * (2 * kGemmMaxStages);
  const uint32_t tempty_bar = tfull_bar + 8;
  const uint32_t drain_bar = tfull_bar + 16;
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
    mbar_init(tfull_bar, 1);
    mbar_init(tempty_bar, 2 * kGemmEpiWarps);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmSW);
    tma_prefetch_desc(&tmSX);
  }
  __syncwarp();
  cluster_sync();  // both CTAs' barriers exist, and both are running
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  grid_dependency_wait();
  if (p.offsets && warp == 2) find_groups(p.offsets, p.groups, start, lane, 8);
  tc_fence_before_sync();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int tiles =
      (p.offsets ? start[p.groups].tiles
                 : p.groups * ((static_cast<int>(p.group_rows) + kBN - 1) / kBN)) * p.m_tiles;

  if (warp == 0) {
    // ---------------------------------------------------------- codes (both CTAs)
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += pairs) {
      const GemmTile tile = gemm_tile<kBN>(t, p, start);
      const int half_n = ((tile.count + 31) & ~31) >> 1;  // rows this CTA holds
      const int boxes = (half_n + p.box_rows - 1) / p.box_rows;
      const bool two = tile.count > kTileRows;
      const uint32_t bytes = kWBytes + static_cast<uint32_t>(boxes * p.box_rows) * kGemmBytesK +
                             S::kScaleStage * (two ? 3 : 2);
      const int w_row = static_cast<int>(tile.group * p.n_out + tile.m * (2 * kGemmM) + rank * kGemmM);
      const int x_row = tile.x_row + rank * half_n;
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!gemm_wait_warp(empty_bar(stage), phase ^ 1u, abort_flag, kWaitEmpty, p)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t w_dst = base + stage * S::kStageBytes;
          const uint32_t x_dst = w_dst + kWBytes;
          const uint32_t full = mapa_shared(full_bar(stage), 0);
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * bytes);
          if (!(p.inject && issued == 0))
            tma_load_2d_pair(w_dst, &tmW, full, kb * kGemmBytesK, w_row);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d_pair(x_dst + b * p.box_rows * kGemmBytesK, &tmX, full, kb * kGemmBytesK,
                             x_row + b * p.box_rows);
        }
        __syncwarp();
        ++issued;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (rank == 0) {  // the even CTA's barriers count both CTAs' bytes
      const uint32_t first = issued > static_cast<uint32_t>(stages) ? issued - stages : 0u;
      for (uint32_t i = first; i < issued; ++i)
        gemm_wait_drain(full_bar(i % stages), (i / stages) & 1u, p.timeout_ns);
    }
  } else if (warp == kGemmRowWarp) {
    // ---------------------------------------------------------- scales (both CTAs)
    // Block i's go where block i - slots' were, whose MMAs have then read theirs
    // from tensor memory too.
    int stage = 0, slot = 0, freed = 0;
    uint32_t freed_phase = 0, issued = 0;
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += pairs) {
      const GemmTile tile = gemm_tile<kBN>(t, p, start);
      int sw = (tile.group * p.w_group_tiles + 2 * tile.m + rank) * p.tile_chunks;
      // each CTA loads one tile of the rows' scales, for both
      int sx = (tile.x_tile + rank) * p.tile_chunks;
      const bool loads_sx = rank == 0 || tile.count > kTileRows;
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (issued >= static_cast<uint32_t>(slots)) {
          if (!gemm_wait_warp(empty_bar(freed), freed_phase, abort_flag, kWaitEmpty, p)) {
            ok = false;
            break;
          }
          if (++freed == stages) {
            freed = 0;
            freed_phase ^= 1u;
          }
        }
        if (elect_one()) {
          const uint32_t dst = scales + slot * S::kSlotBytes;
          const uint32_t full = mapa_shared(full_bar(stage), 0);
          tma_load_2d_pair(dst, &tmSW, full, 0, sw);
          if (loads_sx)
            tma_load_2d_pair_mc(dst + (1 + rank) * S::kScaleStage, &tmSX, full, 0, sx, kBoth);
        }
        __syncwarp();
        sw += kChunks;
        sx += kChunks;
        ++issued;
        if (++stage == stages) stage = 0;
        if (++slot == slots) slot = 0;
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer (even CTA)
    if (rank == 0) {
      int stage = 0, slot = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint64_t w_desc0 = sw128_kmajor_desc(base);
      const uint64_t s_desc0 = scale_desc(scales);
      for (int t = pair; ok && t < tiles; t += pairs) {
        const GemmTile tile = gemm_tile<kBN>(t, p, start);
        const uint32_t idesc = fp4_idesc<kFormat>(2 * kGemmM, (tile.count + 31) & ~31);
        if (!gemm_wait_warp(tempty_bar, acc_phase ^ 1u, abort_flag, kWaitTmemEmpty, p)) break;
        tc_fence_after_sync();
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!gemm_wait_warp(full_bar(stage), phase, abort_flag, kWaitFull, p)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          // No branches in here: leaving out the second tile of scales where the
          // rows have one, or the steps past k, made the issue the bound (170 us
          // at 8192^3 against 166; what is copied for nothing is not used).
          if (elect_one()) {
            const uint64_t at = static_cast<uint64_t>((stage * S::kStageBytes) >> 4);
            const uint64_t s_desc =
                s_desc0 + static_cast<uint64_t>((slot * S::kSlotBytes) >> 4);
            const uint32_t w_cols = tmem + kTmemScales + slot * S::kSlotCols;
            const uint32_t x_cols = w_cols + S::kWCols;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              tmem_copy_scales_pair(w_cols + 4 * c, s_desc + ((c * kChunkBytes) >> 4));
              tmem_copy_scales_pair(x_cols + 8 * c,
                                    s_desc + ((S::kScaleStage + c * kChunkBytes) >> 4));
              tmem_copy_scales_pair(x_cols + 8 * c + 4,
                                    s_desc + ((2 * S::kScaleStage + c * kChunkBytes) >> 4));
            }
            const uint64_t w_desc = w_desc0 + at;
            const uint64_t x_desc = w_desc + (kWBytes >> 4);
#pragma unroll
            for (int s = 0; s < 4; ++s) {  // 64 columns each; past k codes and scales are zero
              const int chunk = kFormat == FP4_NV ? s : s >> 1;
              const int byte = kFormat == FP4_NV ? 0 : (s & 1) * 2;
              umma_fp4_pair<kFormat>(tmem, w_desc + 2u * s, x_desc + 2u * s,
                                     idesc | fp4_idesc_scale_bytes(byte), w_cols + 4 * chunk,
                                     x_cols + 8 * chunk, (kb | s) != 0);
            }
            umma_commit_pair_mc(empty_bar(stage), kBoth);
          }
          __syncwarp();
          if (++slot == slots) slot = 0;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit_pair_mc(tfull_bar, kBoth);
        __syncwarp();
        acc_phase ^= 1u;
      }
      if (elect_one()) umma_commit_pair_mc(drain_bar, 0x1);
      __syncwarp();
      gemm_wait_drain(drain_bar, 0, p.timeout_ns);
      // the last remote arrivals on this CTA's barrier have landed
      gemm_wait_drain(tempty_bar, acc_phase ^ 1u, p.timeout_ns);
    }
  } else {
    // ---------------------------------------------------------- epilogue (both CTAs)
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    uint32_t acc_phase = 0;
    const uint32_t leader_tempty = mapa_shared(tempty_bar, 0);
    for (int t = pair; t < tiles; t += pairs) {
      const GemmTile tile = gemm_tile<kBN>(t, p, start);
      int ok = 0;
      if (lane == 0) ok = gemm_wait(tfull_bar, acc_phase, abort_flag, kWaitTmemFull, p);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after_sync();
      const int64_t n = static_cast<int64_t>(tile.m) * (2 * kGemmM) + rank * kGemmM + q * 32 + lane;
      store_tile<T, 2>(tmem + (static_cast<uint32_t>(q * 32) << 16), half, tile.count, p,
                       p.d + tile.x_row * p.n_out + n, n < p.n_out, [&] {
                         tc_fence_before_sync();
                         __syncwarp();
                         if (lane == 0) mbar_arrive_cluster(leader_tempty);
                       });
      acc_phase ^= 1u;
    }
    zero_tail(p, start);
  }
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace gb300
