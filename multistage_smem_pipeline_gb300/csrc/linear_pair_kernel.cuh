// The products of linear layers over CTA pairs (tcgen05 cta_group::2): tiles of an M
// of 256 and an N of 256 at most.
//
// Each CTA loads its own 128 of M and its half of N, 32 KiB per 64 of the sum where a
// single CTA's 128 x 256 tile takes 48; the even CTA issues, and each accumulates
// its 128 of M in its own tensor memory, in two accumulators by turns.
//
// Barriers as in the other pair kernels: `full` in the even CTA counts both CTAs'
// bytes; `empty` and `tfull` are in both, committed to both; `tempty` in the even
// CTA takes every epilogue warp of both.  grad_w's ragged stages (see linear.cuh)
// are different: each CTA has to zero rows of its own, so their loads count on
// `ragged` of each CTA, and a warp of each zeroes its rows and says so on `ready`
// of the even one; `full` of such a stage is passed at once.
//
// What bounds it: the tensor cores for large dense products (8192^3 577 to 595 us, 0.96 to 0.99
// of the burst rate of cuBLAS; single CTAs 689), below that power; with ragged groups the
// operands of tiles of less than 256 rows, and tiles shared out unevenly (4096 tokens x 8 of 64
// experts, 4096 -> 2048, 376 us for 286 of MMAs at the burst rate).
#pragma once
#include "linear.cuh"

namespace gb300 {

constexpr int kLinPairTile = 256;
constexpr uint32_t kLinPairStage = kLinABytes + kLinPairTile / 2 * kLinK * 2;

template <typename T, int kProduct>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const LinearParams p) {
  constexpr bool kAMn = a_mn(kProduct), kBMn = b_mn(kProduct);
  constexpr bool kWeight = kProduct == LINEAR_GRAD_W;
  constexpr int kM = 2 * kLinM;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.stages;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  constexpr uint16_t kBoth = 0x3;
  const uint32_t bars = base + stages * kLinPairStage;
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

  if (threadIdx.x == 0) {
    linear_begin_early(p);
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(ragged_bar(s), 1);
      mbar_init(ready_bar(s), 2);  // both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 2 * kLinEpiWarps);
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
  cluster_sync();  // both CTAs' barriers exist, and both are running
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * kLinPairTile);
    tmem_relinquish_pair();
  }
  linear_begin(p);
  if (warp == 2) linear_starts(p, start, lane);
  tc_fence_before_sync();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int tiles = linear_tiles<kProduct>(p, start);
  // the N that a CTA holds: half of the tile's, to 16
  const auto half_n = [&](const LinearTile& t) { return (t.n_count + 31) >> 5 << 4; };

  if (warp == 0 || warp == kLinNWarp) {
    // ---------------------------------------------------------- producers (both CTAs)
    LinearRing ring{empty_bar(0), stages, 0, 0, true};
    uint32_t issued = 0, ragged_phase = 0;
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += pairs) {
      const LinearTile tile = linear_tile<kProduct, kM>(t, p, start);
      const int half = half_n(tile);
      const auto loads_of = [&](int r) {
        return linear_loads<kProduct>(tile.m + r * kLinM, tile.m_count - r * kLinM,
                                      tile.n + r * half, half, p);
      };
      const LinearLoads loads = loads_of(rank);
      const uint32_t both_bytes = loads.bytes + loads_of(1 - rank).bytes;
      const int kbs = (tile.k_len + kLinK - 1) / kLinK;
      for (int kb = 0; kb < kbs; ++kb) {
        if (!linear_enter(ring, 1, abort_flag, kLinEmpty, p)) {
          ok = false;
          break;
        }
        const int stage = ring.stage;
        const bool ragged = kWeight && linear_ragged(tile, kb, p);
        ring.step();
        ring.look(1);
        if (elect_one()) {
          const uint32_t full = ragged ? mapa_shared(ragged_bar(stage), rank)
                                       : mapa_shared(full_bar(stage), 0);
          const uint32_t dst = base + stage * kLinPairStage;
          if (warp == 0) {
            if (ragged) mbar_arrive_expect_tx(ragged_bar(stage), loads.bytes);
            if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), ragged ? 0 : both_bytes);
            if (!(p.inject && issued == 0 && rank == 0))
              linear_load_m<kProduct, true>(loads, dst, &tmA, full, kb * kLinK, tile);
          } else {
            linear_load_n<kProduct, true>(loads, dst, &tmB, full, kb * kLinK, tile, p);
          }
        }
        __syncwarp();
        if (ragged) ragged_phase ^= 1u << stage;
        ++issued;
      }
    }
    if (rank == 0) {  // both CTAs' bytes
      const uint32_t first = issued > static_cast<uint32_t>(stages) ? issued - stages : 0u;
      for (uint32_t i = first; i < issued; ++i)
        linear_wait_drain(full_bar(i % stages), (i / stages) & 1u, p.timeout_ns);
    }
    if (kWeight) linear_drain_ragged(ragged_bar(0), stages, ragged_phase, p.timeout_ns);
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------- MMA issuer
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t ready_phase = 0;
    LinearRing ring{full_bar(0), stages, 0, 0, false};
    const uint64_t a_desc0 = linear_desc<kAMn>(base);
    const uint64_t b_desc0 = linear_desc<kBMn>(base + kLinABytes);
    for (int t = pair; t < tiles; t += pairs) {
      const LinearTile tile = linear_tile<kProduct, kM>(t, p, start);
      const uint32_t idesc = linear_idesc<T, kProduct>(kM, 2 * half_n(tile));
      if (!linear_wait_warp(tempty_bar(acc), acc_phase ^ 1u, abort_flag, kLinTmemEmpty, p)) break;
      tc_fence_after_sync();
      if (!linear_multiply<T, kProduct, true, 1>(
              tile, 0, (tile.k_len + kLinK - 1) / kLinK, ring, empty_bar(0), ready_bar(0),
              ready_phase, kLinPairStage >> 4, a_desc0, b_desc0, tmem + acc * kLinPairTile, idesc,
              abort_flag, p))
        break;
      if (elect_one()) umma_commit_pair_mc(tfull_bar(acc), kBoth);
      __syncwarp();
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (elect_one()) umma_commit_pair_mc(drain_bar, 0x1);
    __syncwarp();
    linear_wait_drain(drain_bar, 0, p.timeout_ns);
    // the last remote arrivals on this CTA's barriers have landed
    for (int b = 0; b < 2; ++b) {
      linear_wait_drain(tempty_bar(acc), acc_phase ^ 1u, p.timeout_ns);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  } else if (warp == kLinZeroWarp) {
    // ---------------------------------------------------------- grad_w's ragged stages (both CTAs)
    if (kWeight && p.offsets) {
      int done = 0;  // stages of tiles before
      uint32_t ragged_phase = 0;
      for (int t = pair; t < tiles; t += pairs) {
        const LinearTile tile = linear_tile<kProduct, kM>(t, p, start);
        const int kbs = (tile.k_len + kLinK - 1) / kLinK;
        done += kbs;
        if (kbs == 0 || !linear_ragged(tile, kbs - 1, p)) continue;
        const int stage = (done - 1) % stages;
        if (!linear_wait_warp(ragged_bar(stage), (ragged_phase >> stage) & 1u, abort_flag, kLinFull, p))
          break;
        ragged_phase ^= 1u << stage;
        const uint32_t a = base + stage * kLinPairStage;
        const int valid = tile.k_len - (kbs - 1) * kLinK;
        linear_zero_rows(a, kLinM / 64, valid, lane);
        linear_zero_rows(a + kLinABytes, kLinPairTile / 128, valid, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(ready_bar(stage), 0));
      }
    }
  } else if (warp >= 2) {
    // ---------------------------------------------------------- epilogue (both CTAs)
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    if (kWeight) linear_sum_strips<T>(p, start);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = pair; t < tiles; t += pairs) {
      const LinearTile tile = linear_tile<kProduct, kM>(t, p, start);
      const bool ok = linear_epilogue<T, kProduct>(
          tile, tile.m + rank * kLinM, q, half,
          tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * kLinPairTile, p, lane,
          [&] { return linear_wait_warp(tfull_bar(acc), acc_phase, abort_flag, kLinTmemFull, p); },
          // Nothing in memory goes with it: the accumulator has been read.  With a release
          // the arrival waits until D's stores are performed, and the next tile with it
          // (16 experts, 8192 x 2048 x 4096: tensor cores 47 % busy in grad_w).
          [&] { mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar(acc), 0)); });
      if (!ok) break;
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    linear_zero_tail<kProduct>(p, start);
  }
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync();
  linear_end(p);
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 2 * kLinPairTile);
  }
}

}  // namespace gb300
