// Tokens sorted by expert, their rows gathered in that order, put back with
// weights, and the gradients of both.
//
// With slots p = t * k + j, key(p) the slot's expert (or E when dropped), and
// rows(p) the rank of p by (key, p):
//   dispatch   Y[rows(p)] = X[t]                dX[t] = sum_j dY[rows(p)]
//   combine    O[t] = sum_j w(p) Y[rows(p)]     dY[rows(p)] = w(p) dO[t]
//                                               dw(p) = <dO[t], Y[rows(p)]>
// All but the sort move rows and are bound by memory: each kernel reads its
// inputs once and writes its outputs once, 16 bytes a thread.
#include "moe_common.cuh"

namespace gb300 {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kRowThreads = 256;
constexpr int kSlotThreads = 128;  // a warp per slot

struct RouteParams {
  const int32_t* offsets;
  const int32_t* rows;
  int64_t tokens;
  int32_t top_k, experts, hidden;
};

// ------------------------------------------------------------------ sort
// A cluster of 1 to 8 blocks; the slots are cut into one run per warp, in
// order.  A first walk ranks each slot among its warp's slots of the same key
// (lanes with equal keys by lane, on top of the count of the steps before) and
// leaves the counts per key and warp in shared memory.  These are turned into
// what lies before each warp's slots of a key: within the block by a scan over
// its warps, across blocks from the other blocks' totals (distributed shared
// memory), across keys by a scan over the keys, which is `offsets`.  Ranks and
// keys of a warp's first 256 slots stay in registers; those of later ones wait
// in `rows`.  Everything is read and written once or twice; what bounds the
// sort is latency, hence one launch and few steps: 64 slots take 3.3 us, 32,792
// 7.4 and 65,536 (of 128 experts) 9.2.
__global__ void __launch_bounds__(kSortThreads)
    sort_kernel(int32_t* __restrict__ offsets, int32_t* rows, const int32_t* __restrict__ ids, int n,
                int experts) {
  constexpr int kHeld = 8;            // steps of a warp whose ranks stay in registers
  extern __shared__ int32_t count[];  // [kSortWarps][keys], then [keys] totals, [kSortWarps] sums
  const int keys = experts + 1;
  int32_t* const totals = count + kSortWarps * keys;
  int32_t* const sums = totals + keys;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int blocks = static_cast<int>(gridDim.x);  // one cluster is the grid
  grid_launch_dependents();
  for (int i = threadIdx.x; i < kSortWarps * keys; i += kSortThreads) count[i] = 0;
  const int warps = blocks * kSortWarps;
  const int per_warp = ((n + 32 * warps - 1) / (32 * warps)) * 32;
  const int64_t at = static_cast<int64_t>(rank * kSortWarps + warp) * per_warp;
  const int begin = static_cast<int>(min(at, static_cast<int64_t>(n)));
  const int end = static_cast<int>(min(at + per_warp, static_cast<int64_t>(n)));
  int32_t* const mine = count + warp * keys;
  const auto key_of = [&](int p) {  // past the run: a key of its own
    if (p >= end) return keys;
    const int32_t e = ids[p];
    return (e < 0 || e >= experts) ? experts : e;
  };
  // the rank of a slot among those of its warp so far; lanes with equal keys
  // are found bit by bit (matching them in one instruction took longer:
  // 12.1 against 9.2 us for 65,536 slots of 128 experts)
  const int bits = 32 - __clz(keys);
  const auto place = [&](int key) {
    unsigned same = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
      const bool set = (key >> b) & 1;
      const unsigned with = __ballot_sync(0xffffffffu, set);
      same &= set ? with : ~with;
    }
    const int in = __popc(same & ((1u << lane) - 1u));
    int r = in;
    if (key < keys) r += mine[key];
    __syncwarp();
    if (key < keys && in == 0) mine[key] += __popc(same);
    __syncwarp();
    return r;
  };
  grid_dependency_wait();
  int key[kHeld], held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) key[i] = key_of(begin + 32 * i + lane);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (begin + 32 * i < end) held[i] = place(key[i]);
  for (int p0 = begin + 32 * kHeld; p0 < end; p0 += 32) {
    const int r = place(key_of(p0 + lane));
    if (p0 + lane < end) rows[p0 + lane] = r;
  }
  __syncthreads();
  // over the block's warps: a warp per key, a lane per warp
#pragma unroll 4
  for (int k = warp; k < keys; k += kSortWarps) {
    const int c = count[lane * keys + k];
    int upto = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    count[lane * keys + k] = upto - c;
    if (lane == 31) totals[k] = upto;
  }
  if (blocks > 1) cluster_sync();
  else __syncthreads();
  // over blocks and keys: a thread per key, two of them where there are more
  const int per_thread = (keys + kSortThreads - 1) / kSortThreads;
  int all[2] = {0, 0}, lower[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = static_cast<int>(threadIdx.x) * per_thread + i;
    if (i >= per_thread || k >= keys) continue;
    int c[8];
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      c[b] = 0;
      if (b < blocks)
        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                     : "=r"(c[b])
                     : "r"(mapa_shared(smem_u32(totals + k), b))
                     : "memory");
    }
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      all[i] += c[b];
      if (b < rank) lower[i] += c[b];
    }
  }
  const int total = all[0] + all[1];
  int upto = total;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  if (blocks > 1) cluster_sync();  // the others have read this block's totals
  else __syncthreads();
  int before = lane < warp ? sums[lane] : 0;
#pragma unroll
  for (int d = 16; d; d >>= 1) before += __shfl_xor_sync(0xffffffffu, before, d);
  before += upto - total;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = static_cast<int>(threadIdx.x) * per_thread + i;
    if (i >= per_thread || k >= keys) continue;
    if (rank == 0) offsets[k] = before;
    totals[k] = before + lower[i];  // the first row of this block's slots of the key
    before += all[i];
  }
  __syncthreads();
  const auto put = [&](int p, int k, int r) {
    if (p >= end) return;
    rows[p] = r + mine[k] + totals[k];
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) put(begin + 32 * i + lane, key[i], held[i]);
#pragma unroll 4
  for (int p = begin + 32 * kHeld + lane; p < end; p += 32) put(p, key_of(p), rows[p]);
}

// The slot of each row.
__global__ void __launch_bounds__(kRowThreads)
    pairs_kernel(int32_t* __restrict__ pairs, const int32_t* __restrict__ rows, int n) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int p = static_cast<int>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (p < n) pairs[rows[p]] = p;
}

// ------------------------------------------------------------------ rows out
// Aligned rows: one block per token, whose row is read once and written top_k
// times, so that the traffic is what it has to be.  8192 x 8 rows of 4096 in
// 93 us: 6.5 TB/s, nearly all of it writes.
__global__ void __launch_bounds__(kRowThreads)
    dispatch_kernel(uint16_t* __restrict__ y, const uint16_t* __restrict__ x, int64_t ldx,
                    const RouteParams r) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const int32_t kept = r.offsets[r.experts];
  const int32_t* const rows = r.rows + t * r.top_k;
  const Pack zero = {{0, 0, 0, 0}};
  for (int h = threadIdx.x * 8; h < r.hidden; h += kRowThreads * 8) {
    const Pack v = load8<true>(x + t * ldx, h, r.hidden);
    for (int j = 0; j < r.top_k; ++j) {
      const int32_t row = rows[j];
      store8<true>(y + static_cast<int64_t>(row) * r.hidden, h, r.hidden, row < kept ? v : zero);
    }
  }
}

// Other rows: one warp per slot, as each of a token's rows has windows of its
// own; the token's row comes from cache after the first.  1021 x 6 rows of 1411
// in 5.7 us (7.1 by blocks of a token), of 1408 aligned in 3.8; the shifts and
// the second load of a window are the difference.  Where the slots fill the SMs
// more than once, two windows in flight and more warps do better than four
// (8000 x 2 x 4095: 40.0 against 44.6 us; 1021 x 6 x 1411: 6.7 and 5.7).
template <int kFlight>
__global__ void __launch_bounds__(kSlotThreads)
    dispatch_slots_kernel(uint16_t* __restrict__ y, const uint16_t* __restrict__ x, int64_t ldx,
                          const RouteParams r) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t p = static_cast<int64_t>(blockIdx.x) * (kSlotThreads / 32) + (threadIdx.x >> 5);
  if (p >= r.tokens * r.top_k) return;
  const int32_t row = r.rows[p];
  const bool kept = row < r.offsets[r.experts];
  const uint16_t* const from = x + p / r.top_k * ldx;
  uint16_t* const to = y + static_cast<int64_t>(row) * r.hidden;
  for (int h0 = static_cast<int>(threadIdx.x & 31) * 8 - row_lead(to); h0 < r.hidden;
       h0 += 32 * 8 * kFlight) {
    Pack v[kFlight];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      v[q] = {{0, 0, 0, 0}};
      if (kept && h0 + q * 32 * 8 < r.hidden) v[q] = load8<false>(from, h0 + q * 32 * 8, r.hidden);
    }
#pragma unroll
    for (int q = 0; q < kFlight; ++q)
      if (h0 + q * 32 * 8 < r.hidden) store8<false>(to, h0 + q * 32 * 8, r.hidden, v[q]);
  }
}

// ------------------------------------------------------------------ rows back
// One block per token; kWeighted: the sum takes weights.  The rows of kFlight
// slots are asked for before the first is used; the sum keeps slot order.
// 8192 x 8 rows of 4096 in 89 us: 6.8 TB/s; four in flight against two: 89 and 100.
// Unaligned rows do as well with two as with four (4096 x 8 x 2047: 40 us) as long
// as a thread has at most 40 registers; with 42 it was 48.7.  Two leave room.
template <typename T, bool kAligned, bool kWeighted>
__global__ void __launch_bounds__(kRowThreads, 5)
    combine_kernel(uint16_t* __restrict__ out, const uint16_t* __restrict__ y,
                   const float* __restrict__ weights, const RouteParams r) {
  constexpr int kFlight = kAligned ? 4 : 2;
  __shared__ int32_t s_row[MOE_MAX_TOP_K];
  __shared__ float s_weight[MOE_MAX_TOP_K];
  __shared__ int s_live;
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  if (threadIdx.x < 32) {  // the kept slots, in order
    const int32_t kept = r.offsets[r.experts];
    int live = 0;
    for (int j0 = 0; j0 < r.top_k; j0 += 32) {
      const int j = j0 + static_cast<int>(threadIdx.x);
      const int32_t row = j < r.top_k ? r.rows[t * r.top_k + j] : kept;
      const unsigned in = __ballot_sync(0xffffffffu, row < kept);
      if (row < kept) {
        const int at = live + __popc(in & ((1u << threadIdx.x) - 1u));
        s_row[at] = row;
        if (kWeighted) s_weight[at] = weights[t * r.top_k + j];
      }
      live += __popc(in);
    }
    if (threadIdx.x == 0) s_live = live;
  }
  __syncthreads();
  const int live = s_live;
  uint16_t* const to = out + t * r.hidden;
  const int lead = kAligned ? 0 : row_lead(to);
  for (int h = static_cast<int>(threadIdx.x) * 8 - lead; h < r.hidden; h += blockDim.x * 8) {
    float acc[8] = {};
    for (int j = 0; j < live; j += kFlight) {
      Pack v[kFlight];
#pragma unroll
      for (int q = 0; q < kFlight; ++q)
        if (j + q < live) v[q] = load8<kAligned>(y + static_cast<int64_t>(s_row[j + q]) * r.hidden, h, r.hidden);
#pragma unroll
      for (int q = 0; q < kFlight; ++q) {
        if (j + q >= live) break;
        float f[8];
        unpack<T>(v[q], f);
        const float w = kWeighted ? s_weight[j + q] : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = kWeighted ? fmaf(w, f[i], acc[i]) : acc[i] + f[i];
      }
    }
    store8<kAligned>(to, h, r.hidden, pack<T>(acc));
  }
}

// ------------------------------------------------------------------ gradients of the way back
// One warp per slot: it scales the token's gradient into the slot's row and
// takes its product with the row the slot had.  The warps of a block share
// the token's gradient through L1.  8192 x 8 rows of 4096 in 167 us: 6.8 TB/s.
// Rows that are not aligned need registers for their shifts, and do better with
// fewer windows in flight (8000 x 2 of 4095: 76 us against 87); kMany: and, where
// the slots fill the SMs more than once, with fewer registers and 36 warps on an
// SM instead of 32 (65 us; 300 x 8 of 777, where they do not: 5.2 against 4.4).
template <typename T, bool kAligned, bool kMany>
__global__ void __launch_bounds__(kSlotThreads, kMany ? 9 : 8)
    combine_backward_kernel(uint16_t* __restrict__ grad_y, float* __restrict__ grad_weights,
                            const uint16_t* __restrict__ grad_out, const uint16_t* __restrict__ y,
                            const float* __restrict__ weights, const RouteParams r) {
  constexpr int kFlight = kAligned ? 4 : 2;
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * (kSlotThreads / 32) + (threadIdx.x >> 5);
  if (p >= r.tokens * r.top_k) return;
  const int32_t row = r.rows[p];
  const bool kept = row < r.offsets[r.experts];
  const float w = kept ? weights[p] : 0.0f;
  const uint16_t* const g_row = grad_out + (p / r.top_k) * r.hidden;
  const uint16_t* const y_row = y + static_cast<int64_t>(row) * r.hidden;
  uint16_t* const to = grad_y ? grad_y + static_cast<int64_t>(row) * r.hidden : nullptr;
  const int lead = kAligned || !to ? 0 : row_lead(to);
  float dot = 0.0f;
  for (int h0 = lane * 8 - lead; h0 < r.hidden; h0 += 32 * 8 * kFlight) {
    Pack g[kFlight], v[kFlight];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      const int h = h0 + q * 32 * 8;
      if (h >= r.hidden || !kept) continue;
      if (grad_weights) v[q] = load8<kAligned>(y_row, h, r.hidden);
      g[q] = load8<kAligned>(g_row, h, r.hidden);
    }
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      const int h = h0 + q * 32 * 8;
      if (h >= r.hidden) break;
      float a[8] = {}, b[8];
      if (kept) {
        unpack<T>(g[q], a);
        if (grad_weights) {
          unpack<T>(v[q], b);
          if (!kAligned) {
            clip8(a, h, r.hidden);
            clip8(b, h, r.hidden);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fmaf(a[i], b[i], dot);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= w;
      }
      if (to) store8<kAligned>(to, h, r.hidden, pack<T>(a));
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if (grad_weights && lane == 0) grad_weights[p] = dot;
}

// ------------------------------------------------------------------ host
// Whether every row of these matrices starts on a 16-byte boundary.
bool rows_aligned(std::initializer_list<const void*> ptrs, int64_t hidden, int64_t ld) {
  for (const void* p : ptrs)
    if (!aligned_to(p, 16)) return false;
  return hidden % 8 == 0 && ld % 8 == 0;
}

// The matrices of the row movers: `per_slot` ones have tokens * top_k rows.
struct Operand {
  const void* ptr;
  bool per_slot, written, optional;

  Range range(const moe_routing_t* r, int64_t hidden, int64_t ldx) const {
    uint64_t bytes = 0;
    if (r->tokens > 0 && hidden > 0)
      bytes = per_slot ? static_cast<uint64_t>(r->tokens) * r->top_k * hidden * 2
                       : (static_cast<uint64_t>(r->tokens - 1) * (written ? hidden : ldx) + hidden) * 2;
    return {ptr, bytes, written};
  }
};

// Checks common to them; `weights` and their gradient may be absent.
int check_rows(const Operand& a, const Operand& b, const Operand& c, const void* weights,
               const void* grad_weights, int64_t hidden, int64_t ldx, int type,
               const moe_routing_t* r) {
  int rc = check_routing(r);
  if (rc != GEMM_OK) return rc;
  if (!valid_type(type) || hidden < 0 || hidden > MOE_MAX_HIDDEN || ldx < hidden || ldx > INT_MAX)
    return GEMM_ERR_INVALID_VALUE;
  for (const Operand* o : {&a, &b, &c}) {
    if (r->tokens == 0 || hidden == 0) break;
    if (!o->ptr && !o->optional) return GEMM_ERR_INVALID_VALUE;
  }
  for (const Operand* o : {&a, &b, &c}) {
    if (r->tokens == 0 || hidden == 0) break;
    if (!aligned_to(o->ptr, 2)) return GEMM_ERR_MISALIGNED;
  }
  const uint64_t slots = static_cast<uint64_t>(r->tokens) * r->top_k;
  if (any_overlap({a.range(r, hidden, ldx), b.range(r, hidden, ldx), c.range(r, hidden, ldx),
                   {weights, 4 * slots, false}, {grad_weights, 4 * slots, true}}, r))
    return GEMM_ERR_INVALID_VALUE;
  return GEMM_OK;
}

constexpr Operand kNone{nullptr, false, false, true};

RouteParams route_params(const moe_routing_t* r, int64_t hidden) {
  return RouteParams{r->offsets, r->rows,    r->tokens,
                     r->top_k,   r->experts, static_cast<int32_t>(hidden)};
}

// Blocks of warps, one for each slot.
unsigned slot_blocks(const moe_routing_t* r) {
  constexpr int kWarps = kSlotThreads / 32;
  return static_cast<unsigned>((r->tokens * r->top_k + kWarps - 1) / kWarps);
}

template <bool kWeighted>
int run_combine(void* out, const void* y, const float* weights, int64_t hidden, int type,
                const moe_routing_t* r, cudaStream_t s) {
  int rc = check_rows({out, false, true, false}, {y, true, false, false}, kNone, weights, nullptr,
                      hidden, hidden, type, r);
  if (rc != GEMM_OK) return rc;
  if (r->tokens == 0 || hidden == 0) return GEMM_OK;
  if (kWeighted && !weights) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(weights, 4)) return GEMM_ERR_MISALIGNED;
  int sms = 0;
  if ((rc = require_device(&sms)) != GEMM_OK) return rc;
  const bool wide = rows_aligned({out, y}, hidden, hidden);
  // Smaller blocks where there are blocks enough to fill the SMs several times
  // (4096 x 8 x 2048: 25.5 against 27.1 us; 2000 x 8 x 3001: 32.5 and 26.7, so
  // not yet there), larger ones where a token's row is what one block has to do
  // (16 x 4 x 2048: 1.9 against 2.3); and no threads without a window of the row
  // (1021 x 6 x 1411: 5.9 against 6.5 with 256, 2000 x 4 x 256: 2.5 against 3.6
  // with 128, 8192 x 8 x 1408: 34.9 and 36.4).
  const int64_t most = r->tokens > 16 * sms ? kRowThreads / 2 : kRowThreads;
  const int64_t windows = (hidden + (wide ? 7 : 14)) / 8;
  const int64_t passes = (windows + most - 1) / most;
  const unsigned threads =
      static_cast<unsigned>(((windows + passes - 1) / passes + 31) / 32 * 32);
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(r->tokens)), dim3(threads), 0, s, 1u,
                      static_cast<uint16_t*>(out), static_cast<const uint16_t*>(y), weights,
                      route_params(r, hidden));
  };
  if (type == MOE_F16)
    return wide ? go(combine_kernel<__half, true, kWeighted>)
                : go(combine_kernel<__half, false, kWeighted>);
  return wide ? go(combine_kernel<__nv_bfloat16, true, kWeighted>)
              : go(combine_kernel<__nv_bfloat16, false, kWeighted>);
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" int moe_sort(int32_t* offsets, int32_t* rows, const int32_t* ids, int64_t tokens,
                        int top_k, int experts, void* stream) {
  if (tokens < 0 || top_k < 1 || top_k > MOE_MAX_TOP_K || experts < 1 ||
      experts > MOE_MAX_EXPERTS || tokens > MOE_MAX_SLOTS / top_k)
    return GEMM_ERR_INVALID_VALUE;
  if (!offsets || (tokens > 0 && (!rows || !ids))) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(offsets, 4) || !aligned_to(rows, 4) || !aligned_to(ids, 4))
    return GEMM_ERR_MISALIGNED;
  const uint64_t bytes = static_cast<uint64_t>(tokens) * top_k * 4;
  const uint64_t offset_bytes = (static_cast<uint64_t>(experts) + 1) * 4;
  if (any_overlap({{rows, bytes, true}, {offsets, offset_bytes, true}, {ids, bytes, false}}))
    return GEMM_ERR_INVALID_VALUE;
  int device = 0;
  const int rc = require_device(nullptr, &device);
  if (rc != GEMM_OK) return rc;
  const int n = static_cast<int>(tokens * top_k);
  const auto smem = [](int keys) { return sizeof(int32_t) * ((kSortWarps + 1) * keys + kSortWarps); };
  static std::atomic<uint64_t> granted{0};
  if (!grant_smem(sort_kernel, smem(MOE_MAX_EXPERTS + 1), device, granted)) return GEMM_ERR_CUDA;
  // A slot a thread on one block, and past that a cluster of the largest
  // portable size: a step of a block's warps costs more than the cluster's
  // two meetings: 6,126 slots take 5.8 us on one block and 4.1 on eight, 1,024
  // slots 3.6 and 4.3.
  const unsigned blocks = n <= kSortThreads ? 1 : 8;
  return launch_pdl(sort_kernel, dim3(blocks), dim3(kSortThreads), smem(experts + 1),
                    static_cast<cudaStream_t>(stream), blocks, offsets, rows, ids, n, experts);
}

extern "C" int moe_pairs(int32_t* pairs, const moe_routing_t* r, void* stream) {
  int rc = check_routing(r);
  if (rc != GEMM_OK) return rc;
  if (r->tokens == 0) return GEMM_OK;
  if (!pairs) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(pairs, 4)) return GEMM_ERR_MISALIGNED;
  const int n = static_cast<int>(r->tokens * r->top_k);
  if (any_overlap({{pairs, 4ull * n, true}}, r)) return GEMM_ERR_INVALID_VALUE;
  if ((rc = require_device(nullptr)) != GEMM_OK) return rc;
  return launch_pdl(pairs_kernel, dim3(static_cast<unsigned>((n + kRowThreads - 1) / kRowThreads)),
                    dim3(kRowThreads), 0, static_cast<cudaStream_t>(stream), 1u, pairs, r->rows, n);
}

extern "C" int moe_dispatch(void* y, const void* x, int64_t ldx, int64_t hidden, int type,
                            const moe_routing_t* r, void* stream) {
  int rc = check_rows({y, true, true, false}, {x, false, false, false}, kNone, nullptr, nullptr,
                      hidden, ldx, type, r);
  if (rc != GEMM_OK) return rc;
  if (r->tokens == 0 || hidden == 0) return GEMM_OK;
  int sms = 0;
  if ((rc = require_device(&sms)) != GEMM_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RouteParams p = route_params(r, hidden);
  uint16_t* const to = static_cast<uint16_t*>(y);
  const uint16_t* const from = static_cast<const uint16_t*>(x);
  if (rows_aligned({y, x}, hidden, ldx))
    return launch_pdl(dispatch_kernel, dim3(static_cast<unsigned>(r->tokens)), dim3(kRowThreads), 0,
                      s, 1u, to, from, ldx, p);
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(slot_blocks(r)), dim3(kSlotThreads), 0, s, 1u, to, from, ldx, p);
  };
  return r->tokens * r->top_k > 64 * static_cast<int64_t>(sms) ? go(dispatch_slots_kernel<2>)
                                                               : go(dispatch_slots_kernel<4>);
}

extern "C" int moe_dispatch_backward(void* grad_x, const void* grad_y, int64_t hidden, int type,
                                     const moe_routing_t* r, void* stream) {
  return run_combine<false>(grad_x, grad_y, nullptr, hidden, type, r,
                            static_cast<cudaStream_t>(stream));
}

extern "C" int moe_combine(void* out, const void* y, const float* weights, int64_t hidden,
                           int type, const moe_routing_t* r, void* stream) {
  return run_combine<true>(out, y, weights, hidden, type, r, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_combine_backward(void* grad_y, float* grad_weights, const void* grad_out,
                                    const void* y, const float* weights, int64_t hidden, int type,
                                    const moe_routing_t* r, void* stream) {
  int rc = check_rows({grad_y, true, true, true}, {grad_out, false, false, false},
                      {y, true, false, false}, weights, grad_weights, hidden, hidden, type, r);
  if (rc != GEMM_OK) return rc;
  const int64_t n = r->tokens * r->top_k;
  if (n == 0 || (!grad_y && !grad_weights)) return GEMM_OK;
  if (!weights) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(weights, 4) || !aligned_to(grad_weights, 4)) return GEMM_ERR_MISALIGNED;
  int sms = 0;
  if ((rc = require_device(&sms)) != GEMM_OK) return rc;
  const bool wide = rows_aligned({grad_y, grad_out, y}, hidden, hidden);
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(slot_blocks(r)), dim3(kSlotThreads), 0,
                      static_cast<cudaStream_t>(stream), 1u, static_cast<uint16_t*>(grad_y),
                      grad_weights, static_cast<const uint16_t*>(grad_out),
                      static_cast<const uint16_t*>(y), weights, route_params(r, hidden));
  };
  const bool many = n > 32 * static_cast<int64_t>(sms);
  const auto by_form = [&](auto t) {
    using T = decltype(t);
    if (wide) return go(combine_backward_kernel<T, true, false>);
    return many ? go(combine_backward_kernel<T, false, true>)
                : go(combine_backward_kernel<T, false, false>);
  };
  return type == MOE_F16 ? by_form(__half{}) : by_form(__nv_bfloat16{});
}
