// Pieces shared by the routing, quantisation and 4-bit product translation
// units: argument checks, launches, and conversions of the 16-bit types.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>

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
      r->experts > MOE_MAX_EXPERTS || r->tokens > INT_MAX / r->top_k)
    return GEMM_ERR_INVALID_VALUE;
  if (r->tokens > 0 && (!r->offsets || !r->rows || !r->pairs || !r->ids))
    return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(r->offsets, 4) || !aligned_to(r->rows, 4) || !aligned_to(r->pairs, 4) ||
      !aligned_to(r->ids, 4))
    return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}

// A launch with programmatic dependent launch: the kernel's set-up may overlap
// the end of the one before it in the stream, and every kernel here waits for
// that one (grid_dependency_wait) before its first access to memory.
template <typename... Params, typename... Args>
int launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
               Args... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

inline int require_device(int* sms) {
  int dev = 0;
  DeviceState* st = nullptr;
  const int rc = current_device(&dev, &st);
  if (rc == GEMM_OK && sms) *sms = device_sm_count(st);
  return rc;
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

// N neighbouring 16-bit elements as they are loaded and stored: 8 (16 bytes)
// where rows are 16-byte aligned, else 1.
template <int N>
struct Pack;
template <>
struct Pack<8> {
  uint4 v;
};
template <>
struct Pack<1> {
  uint16_t v;
};

template <typename T, int N>
__device__ __forceinline__ void unpack(const Pack<N>& p, float (&f)[N]) {
  const T* e = reinterpret_cast<const T*>(&p);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = to_float(e[i]);
}

template <typename T, int N>
__device__ __forceinline__ Pack<N> pack(const float (&f)[N]) {
  Pack<N> p;
  T* e = reinterpret_cast<T*>(&p);
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = from_float<T>(f[i]);
  return p;
}

}  // namespace gb300
