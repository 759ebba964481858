// The products of linear layers on single CTAs: tiles of an M of 128 and an N of 32
// to 256.
//
// Inside a CTA, one per SM:
//   warps 0 and 11 -- producers, of M and of N: per 64 of the sum, TMA boxes into a ring
//       (one warp for both took 440 cycles a stage, whatever the tile);
//   warp 1 -- MMA issuer, into two accumulators by turns;
//   warps 2 .. 9 -- epilogue: two warps for each quadrant of lanes, which take
//       32 columns by turns, and store from registers;
//   warp 10 -- grad_w: zeroes the rows of other groups in a sum's last stage.
// The loops of the issuing warps are run by the whole warp, and one lane issues.
//
// kSplit: few tiles.  The CTAs of a cluster share one tile, each taking its part of
// the sum's stages; with all MMAs done, the rings are free, and every CTA writes its
// sums for each other one's share of the chunks into that one's ring, where they
// are added in the order of the parts.  No sum depends on who came first.
//
// What bounds it: with small tiles the issue loop (see linear_multiply), and for few blocks
// a launch's two ends, about 3 us (517 x 1001 x 1411: 12.8 us with its copies).
#pragma once
#include "linear.cuh"

namespace gb300 {

// kBlocks: of 64 of the sum in a stage, 2 for tiles up to 64 (32 x 4096 x 4096 in tiles of 32: 15.2 us
// and 17.2; but 128 x 4096 x 4096 in tiles of 128, for which there are three such stages, 19.3 and 17.8).
template <typename T, int kProduct, bool kSplit, int kBlocks>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_tc(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const LinearParams p) {
  constexpr bool kAMn = a_mn(kProduct), kBMn = b_mn(kProduct);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.stages;
  const uint32_t block_bytes = kLinABytes + p.tile * (kLinK * 2);
  const uint32_t stage_bytes = kBlocks * block_bytes;
  const uint32_t bars = base + stages * stage_bytes;
  const int part = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
  const int first_tile = kSplit ? blockIdx.x / p.split : blockIdx.x;
  const int tile_step = kSplit ? INT_MAX / 4 : gridDim.x;  // kSplit: one tile
  const auto full_bar = [&](int s) { return bars + 8u * s; };
  const auto empty_bar = [&](int s) { return bars + 8u * (kLinMaxStages + s); };
  // grad_w's ragged stages: loaded; and zeroed
  const auto ragged_bar = [&](int s) { return bars + 8u * (2 * kLinMaxStages + s); };
  const auto ready_bar = [&](int s) { return bars + 8u * (3 * kLinMaxStages + s); };
  const auto tfull_bar = [&](int b) { return bars + 8u * (4 * kLinMaxStages + b); };
  const auto tempty_bar = [&](int b) { return bars + 8u * (4 * kLinMaxStages + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (4 * kLinMaxStages + 4);
  uint8_t* const misc = smem + (bars - base) + 8 * kLinBars;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  GroupStart* const start = reinterpret_cast<GroupStart*>(misc + 8);
  // columns between the accumulators: tiles are powers of two
  const uint32_t acc_cols = p.tile;
  const uint32_t tmem_cols = 2 * acc_cols;

  if (threadIdx.x == 0) {
    linear_begin_early(p);
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(ragged_bar(s), 1);
      mbar_init(ready_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), kLinEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (linear_has_sums<kProduct>(p)) {
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmB);
    }
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  linear_begin(p);
  if (warp == 2) linear_starts(p, start, lane);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int tiles = linear_tiles<kProduct>(p, start);
  // this CTA's stages of a tile's sum
  const auto stages_of = [&](const LinearTile& t, int* from, int* end) {
    const int kbs = (t.k_len + kLinK - 1) / kLinK;
    *from = kSplit ? static_cast<int>(static_cast<int64_t>(part) * kbs / p.split) : 0;
    *end = kSplit ? static_cast<int>(static_cast<int64_t>(part + 1) * kbs / p.split) : kbs;
  };

  if (warp == 0 || warp == kLinNWarp) {
    // ---------------------------------------------------------- producers
    LinearRing ring{empty_bar(0), stages, 0, 0, true};
    uint32_t issued = 0, ragged_phase = 0;
    bool ok = true;
    for (int t = first_tile; ok && t < tiles; t += tile_step) {
      const LinearTile tile = linear_tile<kProduct, kLinM>(t, p, start);
      const LinearLoads loads = linear_loads<kProduct>(tile.m, tile.m_count, tile.n, tile.n_count, p);
      int from, end;
      stages_of(tile, &from, &end);
      for (int kb = from; kb < end; kb += kBlocks) {
        if (!linear_enter(ring, 1, abort_flag, kLinEmpty, p)) {
          ok = false;
          break;
        }
        const int blocks = kBlocks == 1 ? 1 : min(kBlocks, end - kb);
        const int stage = ring.stage;
        const bool ragged = kProduct == LINEAR_GRAD_W && linear_ragged(tile, kb + blocks - 1, p);
        ring.step();
        ring.look(1);
        if (elect_one()) {
          // a ragged stage is full at once, and ready once it has landed and is zeroed
          const uint32_t full = ragged ? ragged_bar(stage) : full_bar(stage);
          const uint32_t dst = base + stage * stage_bytes;
          if (warp == 0) {
            mbar_arrive_expect_tx(full, blocks * loads.bytes);
            if (ragged) mbar_arrive(full_bar(stage));
          }
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            if (b >= blocks) break;
            const uint32_t at = dst + b * block_bytes;
            const int k = (kb + b) * kLinK;
            if (warp != 0) linear_load_n<kProduct, false>(loads, at, &tmB, full, k, tile, p);
            else if (!(p.inject && issued == 0))
              linear_load_m<kProduct, false>(loads, at, &tmA, full, k, tile);
          }
        }
        __syncwarp();
        if (ragged) ragged_phase ^= 1u << stage;
        ++issued;
      }
    }
    // every load has landed before the CTA may end
    const uint32_t first = issued > static_cast<uint32_t>(stages) ? issued - stages : 0u;
    for (uint32_t i = first; i < issued; ++i)
      linear_wait_drain(full_bar(i % stages), (i / stages) & 1u, p.timeout_ns);
    if (kProduct == LINEAR_GRAD_W)
      linear_drain_ragged(ragged_bar(0), stages, ragged_phase, p.timeout_ns);
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t ready_phase = 0;
    LinearRing ring{full_bar(0), stages, 0, 0, false};
    const uint64_t a_desc0 = linear_desc<kAMn>(base);
    const uint64_t b_desc0 = linear_desc<kBMn>(base + kLinABytes);
    for (int t = first_tile; t < tiles; t += tile_step) {
      const LinearTile tile = linear_tile<kProduct, kLinM>(t, p, start);
      const uint32_t idesc = linear_idesc<T, kProduct>(kLinM, (tile.n_count + 15) & ~15);
      if (!linear_wait_warp(tempty_bar(acc), acc_phase ^ 1u, abort_flag, kLinTmemEmpty, p)) break;
      tc_fence_after_sync();
      int from, end;
      stages_of(tile, &from, &end);
      if (!linear_multiply<T, kProduct, false, kBlocks>(
              tile, from, end, ring, empty_bar(0), ready_bar(0), ready_phase, block_bytes >> 4,
              a_desc0, b_desc0, tmem + acc * acc_cols, idesc, abort_flag, p))
        break;
      if (elect_one()) umma_commit(tfull_bar(acc));
      __syncwarp();
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (elect_one()) umma_commit(drain_bar);
    __syncwarp();
    linear_wait_drain(drain_bar, 0, p.timeout_ns);
  } else if (warp == kLinZeroWarp) {
    // ---------------------------------------------------------- grad_w's ragged stages
    if (kProduct == LINEAR_GRAD_W && p.offsets) {
      int done = 0;  // stages of tiles before
      uint32_t ragged_phase = 0;
      for (int t = first_tile; t < tiles; t += tile_step) {
        const LinearTile tile = linear_tile<kProduct, kLinM>(t, p, start);
        int from, end;
        stages_of(tile, &from, &end);
        done += (end - from + kBlocks - 1) / kBlocks;
        if (end == from || !linear_ragged(tile, end - 1, p)) continue;
        const int stage = (done - 1) % stages;
        if (!linear_wait_warp(ragged_bar(stage), (ragged_phase >> stage) & 1u, abort_flag, kLinFull, p))
          break;
        ragged_phase ^= 1u << stage;
        const uint32_t a = base + stage * stage_bytes + (end - from - 1) % kBlocks * block_bytes;
        const int valid = tile.k_len - (end - 1) * kLinK;
        linear_zero_rows(a, kLinM / 64, valid, lane);
        linear_zero_rows(a + kLinABytes, p.tile / 64, valid, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ready_bar(stage));
      }
    }
  } else if (!kSplit) {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;               // the lane quadrant this warp may read
    const int half = (warp - 2) >> 2;
    if (kProduct == LINEAR_GRAD_W) linear_sum_strips<T>(p, start);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = first_tile; t < tiles; t += tile_step) {
      const LinearTile tile = linear_tile<kProduct, kLinM>(t, p, start);
      const bool ok = linear_epilogue<T, kProduct>(
          tile, tile.m, q, half, tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * acc_cols, p,
          lane,
          [&] { return linear_wait_warp(tfull_bar(acc), acc_phase, abort_flag, kLinTmemFull, p); },
          [&] { mbar_arrive(tempty_bar(acc)); });
      if (!ok) break;
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    linear_zero_tail<kProduct>(p, start);
  }
  if (kSplit) {
    // ---------------------------------------------------------- parts to their owners
    // Chunk (q, c) is the 4 c + q-th, and CTA u / mine owns the u-th.  Of one's own there
    // is a buffer in the ring for each part.
    const bool live_tile = first_tile < tiles;
    const bool epilogue = warp >= 2 && warp < kLinZeroWarp;
    LinearTile tile = {};
    if (live_tile) tile = linear_tile<kProduct, kLinM>(first_tile, p, start);
    const int mine = max(1, p.tile / 8 / p.split);
    const int chunks = (tile.n_count + 31) >> 5;
    const auto slot = [&](int s, int i) {
      return base + static_cast<uint32_t>(s * mine + i) * kLinBufBytes;
    };
    if (epilogue && kProduct == LINEAR_GRAD_W) linear_sum_strips<T>(p, start);
    int ok = 1;
    if (epilogue && live_tile) ok = linear_wait_warp(tfull_bar(0), 0, abort_flag, kLinTmemFull, p);
    __syncwarp();
    cluster_sync();  // all rings are free
    if (epilogue && live_tile && ok) {
      tc_fence_after_sync();
      int from, end;
      stages_of(tile, &from, &end);
      const int q = warp & 3, half = (warp - 2) >> 2;
      for (int c = half; c < chunks; c += 2) {
        if (linear_chunk<kProduct>(tile, tile.m, q, c, p).live <= 0) continue;
        uint32_t r[32];
        linear_sums(tmem + (static_cast<uint32_t>(q * 32) << 16) + 32 * c, end > from, r);
        const int u = 4 * c + q, owner = u / mine;
        linear_send(mapa_shared(slot(part, u - owner * mine), owner), lane, r);
      }
    }
    __syncwarp();
    cluster_sync();  // all parts have come
    if (epilogue) {
      if (live_tile && ok) {
        for (int i = warp - 2; i < mine; i += kLinEpiWarps) {
          const int u = part * mine + i;
          if (u >= 4 * chunks) break;
          const LinearChunk at = linear_chunk<kProduct>(tile, tile.m, u & 3, u >> 2, p);
          if (at.live <= 0) continue;
          T residual[32];
          linear_residual<T, kProduct>(residual, p, at, lane);
          float v[32];
          linear_add_parts(slot(0, i), p.split, mine * kLinBufBytes, lane, v);
          linear_store<T, kProduct>(v, p, linear_bias<T, kProduct>(p, tile.group, at.col + lane),
                                    residual, at, lane);
        }
      }
      linear_zero_tail<kProduct>(p, start);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  linear_end(p);
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, tmem_cols);
  }
}

}  // namespace gb300
