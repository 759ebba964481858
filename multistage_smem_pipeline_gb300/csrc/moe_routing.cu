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

struct RouteParams {
  const int32_t* offsets;
  const int32_t* rows;
  int64_t tokens;
  int32_t top_k, experts;
  int64_t hidden;
};

// ------------------------------------------------------------------ sort
// One block: each warp owns a run of slots, in order.  Counts per warp and
// key in shared memory, then their sums over (key, warp) in that order: the
// first row of each warp's slots of each key.  A second walk gives each slot
// its place: the lanes of a warp that hold equal keys are ranked by lane.
__global__ void __launch_bounds__(kSortThreads)
    sort_kernel(int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                int32_t* __restrict__ pairs, const int32_t* __restrict__ ids, int n, int experts) {
  extern __shared__ int32_t count[];  // [kSortWarps][experts + 1], then [kSortWarps] sums
  const int keys = experts + 1;
  int32_t* const sums = count + kSortWarps * keys;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  for (int i = threadIdx.x; i < kSortWarps * keys; i += kSortThreads) count[i] = 0;
  __syncthreads();
  grid_dependency_wait();
  const int per_warp = ((n + kSortThreads - 1) / kSortThreads) * 32;
  const int begin = min(warp * per_warp, n), end = min(begin + per_warp, n);
  int32_t* const mine = count + warp * keys;
  const auto key_of = [&](int p) {
    const int32_t e = ids[p];
    return (e < 0 || e >= experts) ? experts : e;
  };
  for (int p = begin + lane; p < end; p += 32) atomicAdd(&mine[key_of(p)], 1);
  __syncthreads();
  // exclusive sums, keys outermost: each thread sums a run of keys
  const int per_thread = (keys + kSortThreads - 1) / kSortThreads;
  const int k0 = min(static_cast<int>(threadIdx.x) * per_thread, keys);
  const int k1 = min(k0 + per_thread, keys);
  int total = 0;
  for (int k = k0; k < k1; ++k)
    for (int w = 0; w < kSortWarps; ++w) total += count[w * keys + k];
  int upto = total;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int before = upto - total;
  for (int w = 0; w < warp; ++w) before += sums[w];
  for (int k = k0; k < k1; ++k) {
    offsets[k] = before;
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = count[w * keys + k];
      count[w * keys + k] = before;
      before += c;
    }
  }
  __syncthreads();
  for (int p0 = begin; p0 < end; p0 += 32) {
    const int p = p0 + lane;
    const int key = p < end ? key_of(p) : keys;  // past the run: a key of its own
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int row = 0;
    if (key < keys) row = mine[key] + rank;
    __syncwarp();
    if (key < keys && rank == 0) mine[key] += __popc(same);
    __syncwarp();
    if (key < keys) {
      rows[p] = row;
      pairs[row] = p;
    }
  }
}

// ------------------------------------------------------------------ rows out
// One block per token: its row is read once and written top_k times.
template <int N>
__global__ void __launch_bounds__(kRowThreads)
    dispatch_kernel(uint16_t* __restrict__ y, const uint16_t* __restrict__ x, int64_t ldx,
                    const RouteParams r) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const int32_t kept = r.offsets[r.experts];
  const int32_t* const rows = r.rows + t * r.top_k;
  for (int64_t h = threadIdx.x * N; h < r.hidden; h += kRowThreads * N) {
    const Pack<N> v = *reinterpret_cast<const Pack<N>*>(x + t * ldx + h);
    for (int j = 0; j < r.top_k; ++j) {
      const int32_t row = rows[j];
      Pack<N> w = v;
      if (row >= kept) std::memset(&w, 0, sizeof(w));
      *reinterpret_cast<Pack<N>*>(y + row * r.hidden + h) = w;
    }
  }
}

// ------------------------------------------------------------------ rows back
// One block per token; kWeighted: the sum takes weights.
template <typename T, int N, bool kWeighted>
__global__ void __launch_bounds__(kRowThreads)
    combine_kernel(uint16_t* __restrict__ out, const uint16_t* __restrict__ y,
                   const float* __restrict__ weights, const RouteParams r) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const int32_t kept = r.offsets[r.experts];
  const int32_t* const rows = r.rows + t * r.top_k;
  for (int64_t h = threadIdx.x * N; h < r.hidden; h += kRowThreads * N) {
    float acc[N] = {};
    for (int j = 0; j < r.top_k; ++j) {
      const int32_t row = rows[j];
      if (row >= kept) continue;
      float v[N];
      unpack<T>(*reinterpret_cast<const Pack<N>*>(y + row * r.hidden + h), v);
      const float w = kWeighted ? weights[t * r.top_k + j] : 1.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = kWeighted ? fmaf(w, v[i], acc[i]) : acc[i] + v[i];
    }
    *reinterpret_cast<Pack<N>*>(out + t * r.hidden + h) = pack<T>(acc);
  }
}

// ------------------------------------------------------------------ gradients of the way back
// One warp per slot: it scales the token's gradient into the slot's row and
// takes its product with the row the slot had.  The warps of a block share
// the token's gradient through L1.
template <typename T, int N>
__global__ void __launch_bounds__(kRowThreads)
    combine_backward_kernel(uint16_t* __restrict__ grad_y, float* __restrict__ grad_weights,
                            const uint16_t* __restrict__ grad_out, const uint16_t* __restrict__ y,
                            const float* __restrict__ weights, const RouteParams r) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (p >= r.tokens * r.top_k) return;
  const int32_t row = r.rows[p];
  const bool kept = row < r.offsets[r.experts];
  const float w = kept ? weights[p] : 0.0f;
  const uint16_t* const g_row = grad_out + (p / r.top_k) * r.hidden;
  const uint16_t* const y_row = y + row * r.hidden;
  float dot = 0.0f;
  for (int64_t h = lane * N; h < r.hidden; h += 32 * N) {
    float g[N] = {}, v[N];
    if (kept) {
      unpack<T>(*reinterpret_cast<const Pack<N>*>(g_row + h), g);
      if (grad_weights) {
        unpack<T>(*reinterpret_cast<const Pack<N>*>(y_row + h), v);
#pragma unroll
        for (int i = 0; i < N; ++i) dot = fmaf(g[i], v[i], dot);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] *= w;
    }
    if (grad_y) *reinterpret_cast<Pack<N>*>(grad_y + row * r.hidden + h) = pack<T>(g);
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

// Checks common to the row movers: `per_slot` matrices have tokens * top_k rows.
struct Operand {
  const void* ptr;
  bool per_slot, written, optional;
};

int check_rows(std::initializer_list<Operand> ops, int64_t hidden, int64_t ldx, int type,
               const moe_routing_t* r) {
  int rc = check_routing(r);
  if (rc != GEMM_OK) return rc;
  if (!valid_type(type) || hidden < 0 || hidden > INT_MAX || ldx < hidden || ldx > INT_MAX)
    return GEMM_ERR_INVALID_VALUE;
  if (r->tokens == 0 || hidden == 0) return GEMM_OK;
  const auto bytes = [&](const Operand& o) {
    if (o.per_slot) return static_cast<uint64_t>(r->tokens) * r->top_k * hidden * 2;
    return (static_cast<uint64_t>(r->tokens - 1) * (o.written ? hidden : ldx) + hidden) * 2;
  };
  for (const Operand& o : ops)
    if (!o.ptr && !o.optional) return GEMM_ERR_INVALID_VALUE;
  for (const Operand& o : ops)
    if (!aligned_to(o.ptr, 2)) return GEMM_ERR_MISALIGNED;
  for (const Operand& o : ops)
    for (const Operand& q : ops)
      if (&o != &q && o.written && o.ptr && q.ptr && overlaps(o.ptr, bytes(o), q.ptr, bytes(q)))
        return GEMM_ERR_INVALID_VALUE;
  return GEMM_OK;
}

RouteParams route_params(const moe_routing_t* r, int64_t hidden) {
  return RouteParams{r->offsets, r->rows, r->tokens, r->top_k, r->experts, hidden};
}

template <bool kWeighted>
int run_combine(void* out, const void* y, const float* weights, int64_t hidden, int type,
                const moe_routing_t* r, cudaStream_t s) {
  int rc = check_rows({{out, false, true, false}, {y, true, false, false}}, hidden, hidden, type, r);
  if (rc != GEMM_OK) return rc;
  if (r->tokens == 0 || hidden == 0) return GEMM_OK;
  if (kWeighted && !weights) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(weights, 4)) return GEMM_ERR_MISALIGNED;
  if ((rc = require_device(nullptr)) != GEMM_OK) return rc;
  const bool wide = rows_aligned({out, y}, hidden, hidden);
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(r->tokens)), dim3(kRowThreads), 0, s,
                      static_cast<uint16_t*>(out), static_cast<const uint16_t*>(y), weights,
                      route_params(r, hidden));
  };
  if (type == MOE_F16)
    return wide ? go(combine_kernel<__half, 8, kWeighted>) : go(combine_kernel<__half, 1, kWeighted>);
  return wide ? go(combine_kernel<__nv_bfloat16, 8, kWeighted>)
              : go(combine_kernel<__nv_bfloat16, 1, kWeighted>);
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" int moe_sort_workspace_bytes(int64_t tokens, int top_k, int experts, uint64_t* bytes) {
  if (!bytes || tokens < 0 || top_k < 1 || top_k > MOE_MAX_TOP_K || experts < 1 ||
      experts > MOE_MAX_EXPERTS || tokens > INT_MAX / top_k)
    return GEMM_ERR_INVALID_VALUE;
  *bytes = 0;
  return GEMM_OK;
}

extern "C" int moe_sort(int32_t* offsets, int32_t* rows, int32_t* pairs, const int32_t* ids,
                        int64_t tokens, int top_k, int experts, void* workspace,
                        uint64_t workspace_bytes, void* stream) {
  uint64_t need = 0;
  int rc = moe_sort_workspace_bytes(tokens, top_k, experts, &need);
  if (rc != GEMM_OK) return rc;
  if (!offsets || (tokens > 0 && (!rows || !pairs || !ids))) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(offsets, 4) || !aligned_to(rows, 4) || !aligned_to(pairs, 4) ||
      !aligned_to(ids, 4))
    return GEMM_ERR_MISALIGNED;
  if (need > 0 && (!workspace || workspace_bytes < need)) return GEMM_ERR_INVALID_VALUE;
  if (need > 0 && !aligned_to(workspace, 16)) return GEMM_ERR_MISALIGNED;
  if ((rc = require_device(nullptr)) != GEMM_OK) return rc;
  const int n = static_cast<int>(tokens * top_k);
  const size_t smem = sizeof(int32_t) * kSortWarps * (experts + 2);
  if (cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(sizeof(int32_t) * kSortWarps * (MOE_MAX_EXPERTS + 2))) !=
      cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return launch_pdl(sort_kernel, dim3(1), dim3(kSortThreads), smem,
                    static_cast<cudaStream_t>(stream), offsets, rows, pairs, ids, n, experts);
}

extern "C" int moe_dispatch(void* y, const void* x, int64_t ldx, int64_t hidden, int type,
                            const moe_routing_t* r, void* stream) {
  int rc = check_rows({{y, true, true, false}, {x, false, false, false}}, hidden, ldx, type, r);
  if (rc != GEMM_OK) return rc;
  if (r->tokens == 0 || hidden == 0) return GEMM_OK;
  if ((rc = require_device(nullptr)) != GEMM_OK) return rc;
  const dim3 grid(static_cast<unsigned>(r->tokens)), block(kRowThreads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RouteParams p = route_params(r, hidden);
  return rows_aligned({y, x}, hidden, ldx)
             ? launch_pdl(dispatch_kernel<8>, grid, block, 0, s, static_cast<uint16_t*>(y),
                          static_cast<const uint16_t*>(x), ldx, p)
             : launch_pdl(dispatch_kernel<1>, grid, block, 0, s, static_cast<uint16_t*>(y),
                          static_cast<const uint16_t*>(x), ldx, p);
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
  int rc = check_rows({{grad_y, true, true, true},
                       {grad_out, false, false, false},
                       {y, true, false, false}},
                      hidden, hidden, type, r);
  if (rc != GEMM_OK) return rc;
  const int64_t n = r->tokens * r->top_k;
  if (n == 0 || (!grad_y && !grad_weights)) return GEMM_OK;
  if (!weights) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(weights, 4) || !aligned_to(grad_weights, 4)) return GEMM_ERR_MISALIGNED;
  if ((rc = require_device(nullptr)) != GEMM_OK) return rc;
  const bool wide = rows_aligned({grad_y, grad_out, y}, hidden, hidden);
  const int64_t blocks = (n + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kRowThreads), 0,
                      static_cast<cudaStream_t>(stream), static_cast<uint16_t*>(grad_y),
                      grad_weights, static_cast<const uint16_t*>(grad_out),
                      static_cast<const uint16_t*>(y), weights, route_params(r, hidden));
  };
  if (type == MOE_F16)
    return wide ? go(combine_backward_kernel<__half, 8>) : go(combine_backward_kernel<__half, 1>);
  return wide ? go(combine_backward_kernel<__nv_bfloat16, 8>)
              : go(combine_backward_kernel<__nv_bfloat16, 1>);
}
