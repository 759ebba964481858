// Pieces shared by the routing, quantisation and 4-bit product translation
// units: argument checks, launches, and conversions of the 16-bit types.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "host.cuh"
#include "moe_fp4.h"
#include "ptx.cuh"

namespace gb300 {

// ------------------------------------------------------------------ host
inline bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

inline bool valid_type(int type) { return type == MOE_F16 || type == MOE_BF16; }

// The routing's own fields: sizes in range, and the arrays that a call reads.
inline int check_routing(const moe_routing_t* r) {
  if (!r || r->tokens < 0 || r->top_k < 1 || r->top_k > MOE_MAX_TOP_K || r->experts < 1 ||
      r->experts > MOE_MAX_EXPERTS || r->tokens > MOE_MAX_SLOTS / r->top_k)
    return GEMM_ERR_INVALID_VALUE;
  if (r->tokens > 0 && (!r->offsets || !r->rows || !r->ids))
    return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(r->offsets, 4) || !aligned_to(r->rows, 4) || !aligned_to(r->ids, 4))
    return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}

// An array of a call, and whether the call writes it.
struct Range {
  const void* ptr;
  uint64_t bytes;
  bool written;
};

// Whether a written array overlaps any other, the routing's (which later calls
// still read) among them.  Absent and empty ones overlap nothing.
inline bool any_overlap(std::initializer_list<Range> arrays, const moe_routing_t* r = nullptr) {
  const auto meet = [](const Range& a, const Range& b) {
    return a.ptr && b.ptr && a.bytes && b.bytes && overlaps(a.ptr, a.bytes, b.ptr, b.bytes);
  };
  Range of_routing[2] = {};
  if (r) {
    of_routing[0] = {r->offsets, (static_cast<uint64_t>(r->experts) + 1) * 4, false};
    of_routing[1] = {r->rows, static_cast<uint64_t>(r->tokens) * r->top_k * 4, false};
  }
  for (const Range& a : arrays) {
    if (!a.written) continue;
    for (const Range& b : arrays)
      if (&a != &b && meet(a, b)) return true;
    for (const Range& b : of_routing)
      if (meet(a, b)) return true;
  }
  return false;
}

// A launch with programmatic dependent launch: the kernel's set-up may overlap
// the end of the one before it in the stream, and every kernel here waits for
// that one (grid_dependency_wait) before its first access to memory.
// `cluster` blocks form a cluster.
template <typename... Params, typename... Args>
int launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
               unsigned cluster, Args... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

// The current device, checked; its SM count and number where asked for.
inline int require_device(int* sms, int* device = nullptr) {
  int dev = 0;
  DeviceState* st = nullptr;
  const int rc = current_device(&dev, &st);
  if (rc == GEMM_OK && sms) *sms = device_sm_count(st);
  if (device) *device = dev;
  return rc;
}

// Lets a kernel have `bytes` of dynamic shared memory on a device, once for
// each; `done` has a bit per device (the library knows up to 64).
template <typename Kernel>
bool grant_smem(Kernel kernel, size_t bytes, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = uint64_t{1} << device;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes)) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

// ------------------------------------------------------------------ device
template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }

// Eight neighbouring 16-bit elements.
struct alignas(16) Pack {
  uint32_t w[4];
};

template <typename T>
__device__ __forceinline__ void unpack(const Pack& p, float (&f)[8]) {
  const T* const e = reinterpret_cast<const T*>(&p);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_float(e[i]);
}

template <typename T>
__device__ __forceinline__ Pack pack(const float (&f)[8]) {
  Pack p;
  T* const e = reinterpret_cast<T*>(&p);
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_float<T>(f[i]);
  return p;
}

// Rows that do not start on 16-byte boundaries.  A row is walked in windows of
// eight elements that are aligned where they are stored; the first begins
// `lead` elements before the row, and only the first and the last windows hold
// elements outside it.
__device__ __forceinline__ int row_lead(const uint16_t* row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) >> 1;
}

// The 16 bytes from byte `off` (even, below 16) of the 32 of two words on.
__device__ __forceinline__ Pack shift8(const uint4& lo, const uint4& hi, uint32_t off) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  Pack p;
#pragma unroll
  for (int i = 0; i < 4; ++i) p.w[i] = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
  return p;
}

// Elements [e, e + 8) of a row of n.  Unaligned: the one or two 16-byte words
// that hold them, shifted into place; a word without an element of the row in
// it is not read, and what stands outside the row is undefined.
template <bool kAligned>
__device__ __forceinline__ Pack load8(const uint16_t* row, int e, int n) {
  if (kAligned) return *reinterpret_cast<const Pack*>(row + e);
  const uintptr_t start = reinterpret_cast<uintptr_t>(row);
  const uintptr_t at = start + 2 * static_cast<intptr_t>(e);  // may lie before the row
  const uintptr_t word = at & ~static_cast<uintptr_t>(15);
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  if (word + 16 > start && word < start + 2 * static_cast<uintptr_t>(n))
    lo = *reinterpret_cast<const uint4*>(word);
  const uint32_t off = static_cast<uint32_t>(at & 15);
  if (off == 0) {  // for the whole row: it is aligned as the windows are
    Pack p;
    *reinterpret_cast<uint4*>(&p) = lo;
    return p;
  }
  if (word + 16 < start + 2 * static_cast<uintptr_t>(n))
    hi = *reinterpret_cast<const uint4*>(word + 16);
  return shift8(lo, hi, off);
}

// The same window to a row that it is aligned in; elements outside are left out.
template <bool kAligned>
__device__ __forceinline__ void store8(uint16_t* row, int e, int n, const Pack& p) {
  if (kAligned || (e >= 0 && e + 8 <= n)) {
    *reinterpret_cast<Pack*>(row + e) = p;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i >= 0 && e + i < n) row[e + i] = static_cast<uint16_t>(p.w[i >> 1] >> (16 * (i & 1)));
}

// Zeroes what a window holds outside a row of n elements.
__device__ __forceinline__ void clip8(float (&f)[8], int e, int n) {
  if (e >= 0 && e + 8 <= n) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i < 0 || e + i >= n) f[i] = 0.0f;
}

}  // namespace gb300
