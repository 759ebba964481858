// Host pieces of the kernels that load by TMA: the driver's encoder of tensor
// maps, and the error word that each stream's launches report to.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "gemm_tn_f16.h"

namespace gb300 {

constexpr int kErrorWords = 64;

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline int get_encoder(EncodeTiledFn* encode) {
  static std::atomic<EncodeTiledFn> known{nullptr};
  *encode = known.load(std::memory_order_acquire);
  if (*encode) return GEMM_OK;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || fn == nullptr) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  *encode = reinterpret_cast<EncodeTiledFn>(fn);
  known.store(*encode, std::memory_order_release);
  return GEMM_OK;
}

// Index of a stream's error word: 0 for the legacy default stream, one each
// for the first 63 others, then shared by a hash.
inline int error_index(cudaStream_t s) {
  static std::mutex mu;
  static uintptr_t streams[kErrorWords];
  static int used = 1;
  const uintptr_t h = reinterpret_cast<uintptr_t>(s);
  if (h == 0) return 0;
  std::lock_guard<std::mutex> lk(mu);
  for (int i = 1; i < used; ++i)
    if (streams[i] == h) return i;
  if (used < kErrorWords) {
    streams[used] = h;
    return used++;
  }
  return 1 + static_cast<int>((h >> 4) % (kErrorWords - 1));
}

}  // namespace gb300
