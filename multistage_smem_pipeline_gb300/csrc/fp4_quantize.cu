// Quantisation to 4-bit blocks, and back.
//
// Each thread takes 16 neighbouring elements (a block of FP4_NV, half a block
// of FP4_MX).  Both kernels read and write every element once and are bound
// by memory: 2 bytes in and 1/2 + 1/16 (1/32) out per element, or the reverse.
#include "fp4.cuh"

namespace gb300 {
namespace {

constexpr int kSegment = 16;                            // elements a thread takes
constexpr int kTileSegments = kStageCols / kSegment;    // 16 of them across a tile's 256 columns
constexpr int kThreads = 256;

// 16 elements of a row from column c on; zeros from `cols` on.  kVec: the row
// is 16-byte aligned.
template <typename T, bool kVec>
__device__ __forceinline__ void load_segment(const uint16_t* row, int64_t c, int64_t cols,
                                             float (&f)[kSegment]) {
  if (kVec && c + kSegment <= cols) {
    const uint4* const q = reinterpret_cast<const uint4*>(row + c);
    const uint4 v[2] = {q[0], q[1]};
    const T* const e = reinterpret_cast<const T*>(v);
#pragma unroll
    for (int i = 0; i < kSegment; ++i) f[i] = to_float(e[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < kSegment; ++i) {
    f[i] = 0.0f;
    if (c + i < cols) f[i] = to_float(reinterpret_cast<const T*>(row)[c + i]);
  }
}

struct Segment {
  uint2 codes;
  uint32_t scale;  // byte
};

// f / (scale 2^exponent) to codes.  FP4_MX: called by whole warps, the two
// threads of a block being neighbours.
//
// The quotient must round to E2M1 as the exact one does, ties included, and
// x times the rounded reciprocal does not always: for scales of significand
// 13/8 to 15/8 some exact ties move.  One residual step (Markstein) puts it
// right: q = x r, q + r (x - q s).  Checked for every fp16 and bf16 value
// against every scale.
template <int kFormat>
__device__ __forceinline__ Segment quantize_segment(float (&f)[kSegment], const Fp4View& v) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kSegment; ++i) {
    if (kFormat == FP4_NV) f[i] *= v.down;
    // as bits, so that a NaN is larger than everything
    top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(f[i]) & 0x7fffffffu));
  }
  Segment s;
  if (kFormat == FP4_NV) {
    const bool finite = __float_as_uint(top) < 0x7f800000u;
    s.scale = finite ? to_e4m3(__fdiv_rn(top, 6.0f)) : kNanE4M3;
    const float step = finite ? from_e4m3(s.scale) : 0.0f;
    const float inv = step > 0.0f ? __frcp_rn(step) : 0.0f;
#pragma unroll
    for (int i = 0; i < kSegment; ++i) {
      const float q = f[i] * inv;
      f[i] = finite ? fmaf(fmaf(-q, step, f[i]), inv, q) : 0.0f;
    }
  } else {
    top = __uint_as_float(max(__float_as_uint(top),
                              __shfl_xor_sync(0xffffffffu, __float_as_uint(top), 1)));
    const int field = static_cast<int>(__float_as_uint(top) >> 23);
    s.scale = field == 0xff ? kNanE8M0 : static_cast<uint32_t>(max(field - 2, 0));
    const float inv = field == 0xff ? 0.0f : __uint_as_float((254u - s.scale) << 23);
#pragma unroll
    for (int i = 0; i < kSegment; ++i) f[i] = field == 0xff ? 0.0f : f[i] * inv;
  }
  s.codes = make_uint2(to_e2m1(f), to_e2m1(f + 8));
  return s;
}

// A block per 128-row tile and 256 columns: thread i takes segment i % 16 of
// rows i / 16 + 16 n.  The tile's scales are put together in shared memory and
// written in one piece.
template <typename T, int kFormat, bool kVec>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const Fp4View v, const uint16_t* __restrict__ x, int64_t ldx) {
  constexpr int kBytes = chunks_per_stage(kFormat) * kChunkBytes;
  __shared__ __align__(16) uint8_t scales[kBytes];
  grid_launch_dependents();
  const TileRows t = tile_rows(v, blockIdx.x);
  for (int i = threadIdx.x; i < kBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(scales)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  grid_dependency_wait();
  const int seg = threadIdx.x % kTileSegments;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kStageCols + seg * kSegment;
  for (int r0 = 0; r0 < t.count; r0 += kThreads / kTileSegments) {
    const int r = r0 + threadIdx.x / kTileSegments;
    const bool live = r < t.count;
    float f[kSegment];
    load_segment<T, kVec>(x + (t.row + r) * ldx, c, live ? v.cols : 0, f);
    const Segment s = quantize_segment<kFormat>(f, v);
    if (!live) continue;
    if (c / 2 < v.pitch)
      *reinterpret_cast<uint2*>(v.codes + (t.row + r) * v.pitch + c / 2) = s.codes;
    if (c < v.cols) scales[scale_at(r, kFormat == FP4_NV ? seg : seg >> 1)] = s.scale;
  }
  __syncthreads();
  uint8_t* const to = v.scales + t.tile * v.tile_bytes + static_cast<int64_t>(blockIdx.y) * kBytes;
  for (int i = threadIdx.x; i < kBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(scales)[i];
}

// A block per token and up to 4096 columns: quantised once, written to the
// row of each of its slots.  Neighbouring threads join the four scale bytes
// of a chunk.
template <typename T, int kFormat, bool kVec>
__global__ void __launch_bounds__(kThreads)
    quantize_routed_kernel(const Fp4View v, const uint16_t* __restrict__ x, int64_t ldx,
                           const int32_t* __restrict__ rows, const int32_t* __restrict__ ids,
                           int top_k) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t token = blockIdx.x;
  const int64_t seg = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x;
  const int64_t c = seg * kSegment;
  const int64_t cols256 = col_stages(v.cols) * kStageCols;
  float f[kSegment];
  load_segment<T, kVec>(x + token * ldx, c, v.cols, f);
  const Segment s = quantize_segment<kFormat>(f, v);
  // bytes of the chunk's four blocks, in every thread
  constexpr int kPerBlock = kFormat == FP4_NV ? 1 : 2;
  uint32_t word = (c < v.cols ? s.scale : 0u) << (8 * (seg / kPerBlock & 3));
  if (kFormat == FP4_MX && (seg & 1)) word = 0;
#pragma unroll
  for (int d = 1; d < 4 * kPerBlock; d <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, d);
  if (c >= cols256) return;
  const int32_t kept = v.offsets[v.groups];
  for (int j = 0; j < top_k; ++j) {
    const int32_t row = rows[token * top_k + j];
    if (row >= kept) continue;
    if (c / 2 < v.pitch)
      *reinterpret_cast<uint2*>(v.codes + row * v.pitch + c / 2) = s.codes;
    if (seg % (4 * kPerBlock) == 0) {
      const int32_t e = ids[token * top_k + j];
      const int32_t first = v.offsets[e];
      const int64_t tile = first / kTileRows + e + (row - first) / kTileRows;
      *reinterpret_cast<uint32_t*>(v.scales + tile * v.tile_bytes +
                                   scale_at((row - first) % kTileRows,
                                            static_cast<int>(seg / kPerBlock))) = word;
    }
  }
}

template <typename T, int kFormat, bool kVec>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(uint16_t* __restrict__ y, const Fp4View v) {
  constexpr int kBytes = chunks_per_stage(kFormat) * kChunkBytes;
  __shared__ __align__(16) uint8_t scales[kBytes];
  grid_launch_dependents();
  grid_dependency_wait();
  const TileRows t = tile_rows(v, blockIdx.x);
  if (t.count == 0) return;
  if (t.tile >= 0) {
    const uint8_t* const from =
        v.scales + t.tile * v.tile_bytes + static_cast<int64_t>(blockIdx.y) * kBytes;
    for (int i = threadIdx.x; i < kBytes / 16; i += kThreads)
      reinterpret_cast<uint4*>(scales)[i] = reinterpret_cast<const uint4*>(from)[i];
  }
  __syncthreads();
  const int seg = threadIdx.x % kTileSegments;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kStageCols + seg * kSegment;
  if (c >= v.cols) return;
  for (int r = threadIdx.x / kTileSegments; r < t.count; r += kThreads / kTileSegments) {
    float f[kSegment] = {};
    if (t.tile >= 0) {
      const uint2 codes = *reinterpret_cast<const uint2*>(v.codes + (t.row + r) * v.pitch + c / 2);
      from_e2m1(codes.x, f);
      from_e2m1(codes.y, f + 8);
      const uint32_t byte = scales[scale_at(r, kFormat == FP4_NV ? seg : seg >> 1)];
      const float step = scale_value<kFormat>(byte) * (kFormat == FP4_NV ? v.up : 1.0f);
#pragma unroll
      for (int i = 0; i < kSegment; ++i) f[i] *= step;
    }
    uint16_t* const row = y + (t.row + r) * v.cols;
    if (kVec && c + kSegment <= v.cols) {
      uint4 o[2];
      T* const e = reinterpret_cast<T*>(o);
#pragma unroll
      for (int i = 0; i < kSegment; ++i) e[i] = from_float<T>(f[i]);
      reinterpret_cast<uint4*>(row + c)[0] = o[0];
      reinterpret_cast<uint4*>(row + c)[1] = o[1];
    } else {
#pragma unroll
      for (int i = 0; i < kSegment; ++i)
        if (c + i < v.cols) reinterpret_cast<T*>(row)[c + i] = from_float<T>(f[i]);
    }
  }
}

// Calls f(T{}, format, vec) with the types and constants of this call.
template <typename F>
int dispatch_forms(int type, int format, bool vec, F f) {
  const auto by_vec = [&](auto t, auto fmt) {
    return vec ? f(t, fmt, std::true_type{}) : f(t, fmt, std::false_type{});
  };
  const auto by_format = [&](auto t) {
    return format == FP4_NV ? by_vec(t, std::integral_constant<int, FP4_NV>{})
                            : by_vec(t, std::integral_constant<int, FP4_MX>{});
  };
  return type == MOE_F16 ? by_format(__half{}) : by_format(__nv_bfloat16{});
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" int fp4_code_bytes(int64_t rows, int64_t cols, uint64_t* bytes) {
  if (!bytes || !fits(rows, cols)) return GEMM_ERR_INVALID_VALUE;
  *bytes = static_cast<uint64_t>(rows) * code_pitch(cols);
  return GEMM_OK;
}

extern "C" int fp4_scale_bytes(int64_t rows, int64_t cols, int format, int groups, int by_offsets,
                               uint64_t* bytes) {
  if (!bytes || !fits(rows, cols) || check_format(format) != GEMM_OK || groups < 1 ||
      (by_offsets != 0 && by_offsets != 1) || (by_offsets && groups > MOE_MAX_EXPERTS) ||
      (!by_offsets && rows % groups != 0))
    return GEMM_ERR_INVALID_VALUE;
  *bytes = static_cast<uint64_t>(tile_count(rows, groups, by_offsets != 0)) *
           tile_bytes(cols, format);
  return GEMM_OK;
}

extern "C" int fp4_quantize(const fp4_matrix_t* out, const void* x, int64_t ldx, int type,
                            const moe_routing_t* routing, void* stream) {
  bool any = false;
  int rc = check_matrix(out, &any);
  if (rc != GEMM_OK) return rc;
  if (!valid_type(type) || ldx < out->cols || ldx > INT_MAX) return GEMM_ERR_INVALID_VALUE;
  int64_t x_rows = out->rows;
  if (routing) {
    if ((rc = check_routing(routing)) != GEMM_OK) return rc;
    if (out->offsets != routing->offsets || out->groups != routing->experts ||
        out->rows != routing->tokens * routing->top_k)
      return GEMM_ERR_INVALID_VALUE;
    x_rows = routing->tokens;
  } else if (out->offsets) {
    return GEMM_ERR_INVALID_VALUE;
  }
  if (!any) return GEMM_OK;
  if (!x) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(x, 2)) return GEMM_ERR_MISALIGNED;
  const uint64_t xbytes = (static_cast<uint64_t>(x_rows - 1) * ldx + out->cols) * 2;
  if (overlaps(x, xbytes, out->codes, code_bytes(out)) ||
      overlaps(x, xbytes, out->scales, scale_bytes(out)) ||
      overlaps(out->codes, code_bytes(out), out->scales, scale_bytes(out)))
    return GEMM_ERR_INVALID_VALUE;
  if ((rc = require_device(nullptr)) != GEMM_OK) return rc;
  const Fp4View v = view_of(out);
  const uint16_t* const xp = static_cast<const uint16_t*>(x);
  const bool vec = aligned_to(x, 16) && ldx % 8 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dispatch_forms(type, out->format, vec, [&](auto t, auto fmt, auto wide) {
    using T = decltype(t);
    if (routing) {
      const int64_t segments = col_stages(out->cols) * kTileSegments;
      const dim3 grid(static_cast<unsigned>(x_rows),
                      static_cast<unsigned>((segments + kThreads - 1) / kThreads));
      return launch_pdl(quantize_routed_kernel<T, fmt(), wide()>, grid, dim3(kThreads), 0, s, v, xp,
                        ldx, routing->rows, routing->ids, routing->top_k);
    }
    const dim3 grid(static_cast<unsigned>(tile_count(out->rows, out->groups, false)),
                    static_cast<unsigned>(col_stages(out->cols)));
    return launch_pdl(quantize_kernel<T, fmt(), wide()>, grid, dim3(kThreads), 0, s, v, xp, ldx);
  });
}

extern "C" int fp4_dequantize(void* y, int type, const fp4_matrix_t* in, void* stream) {
  bool any = false;
  int rc = check_matrix(in, &any);
  if (rc != GEMM_OK) return rc;
  if (!valid_type(type)) return GEMM_ERR_INVALID_VALUE;
  if (!any) return GEMM_OK;
  if (!y) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(y, 2)) return GEMM_ERR_MISALIGNED;
  const uint64_t ybytes = static_cast<uint64_t>(in->rows) * in->cols * 2;
  if (overlaps(y, ybytes, in->codes, code_bytes(in)) ||
      overlaps(y, ybytes, in->scales, scale_bytes(in)))
    return GEMM_ERR_INVALID_VALUE;
  if ((rc = require_device(nullptr)) != GEMM_OK) return rc;
  const Fp4View v = view_of(in);
  const bool vec = aligned_to(y, 16) && in->cols % 8 == 0;
  const bool by_offsets = in->offsets != nullptr;
  const dim3 grid(
      static_cast<unsigned>(tile_count(in->rows, in->groups, by_offsets) + (by_offsets ? 1 : 0)),
      static_cast<unsigned>(col_stages(in->cols)));
  return dispatch_forms(type, in->format, vec, [&](auto t, auto fmt, auto wide) {
    using T = decltype(t);
    return launch_pdl(dequantize_kernel<T, fmt(), wide()>, grid, dim3(kThreads), 0,
                      static_cast<cudaStream_t>(stream), static_cast<uint16_t*>(y), v);
  });
}
