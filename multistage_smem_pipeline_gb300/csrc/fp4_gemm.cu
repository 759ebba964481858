// D[r][n] = alpha * sum_k a[r][k] b[g(r)][n][k] on 4-bit matrices.
#include <cmath>

#include "fp4.cuh"

namespace gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;   // rows and outputs of a block's tile
constexpr int kDepth = 64;  // columns per step

// value of element k of a row: code times block scale
template <int kFormat>
__device__ __forceinline__ void decode_row(const Fp4View& v, int64_t row, int64_t tile, int r,
                                           int64_t k, float (&f)[16]) {
  const uint2 codes = *reinterpret_cast<const uint2*>(v.codes + row * v.pitch + k / 2);
  from_e2m1(codes.x, f);
  from_e2m1(codes.y, f + 8);
  const float step = scale_value<kFormat>(
      v.scales[tile * v.tile_bytes + scale_at(r, static_cast<int>(k / block_size(kFormat)))]);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] *= step;
}

// A block per 64 x 64 tile of D, decoded into shared memory 64 columns at a
// time; each thread sums 4 x 4 outputs in fp32.
template <typename T, int kFormat>
__global__ void __launch_bounds__(kThreads)
    fp4_gemm_kernel(uint16_t* __restrict__ d, const Fp4View a, const Fp4View b, float alpha) {
  __shared__ float sa[kTile][kDepth + 1], sb[kTile][kDepth + 1];
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t n_out = b.group_rows;
  int64_t row, end, first;  // this tile's rows, and its group's first row
  int g;
  if (a.offsets) {
    g = find_group(a.offsets, a.groups, kTile, blockIdx.x);
    first = a.offsets[g];
    end = g < a.groups ? a.offsets[g + 1] : a.rows;
    row = first + (blockIdx.x - (first / kTile + g)) * static_cast<int64_t>(kTile);
  } else {
    const int64_t per = (a.group_rows + kTile - 1) / kTile;
    g = static_cast<int>(blockIdx.x / per);
    first = g * a.group_rows;
    end = first + a.group_rows;
    row = first + (blockIdx.x - g * per) * kTile;
  }
  const int count = static_cast<int>(max(min(static_cast<int64_t>(kTile), end - row), int64_t{0}));
  if (count == 0) return;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const bool live = g < a.groups;
  const int64_t a_tile0 = a.offsets ? first / kTileRows + g
                                    : g * ((a.group_rows + kTileRows - 1) / kTileRows);
  const int64_t b_tile0 = g * ((n_out + kTileRows - 1) / kTileRows);
  float acc[4][4] = {};
  const int lr = threadIdx.x >> 2, lk = (threadIdx.x & 3) * 16;
  for (int64_t k0 = 0; live && k0 < a.cols; k0 += kDepth) {
    const int64_t k = k0 + lk;
    float f[16] = {}, h[16] = {};
    if (lr < count && k / 2 < a.pitch) {
      const int64_t in = row + lr - first;
      decode_row<kFormat>(a, row + lr, a_tile0 + in / kTileRows, static_cast<int>(in % kTileRows), k, f);
    }
    if (n0 + lr < n_out && k / 2 < b.pitch)
      decode_row<kFormat>(b, g * n_out + n0 + lr, b_tile0 + (n0 + lr) / kTileRows,
                          static_cast<int>((n0 + lr) % kTileRows), k, h);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      sa[lr][lk + i] = f[i];
      sb[lr][lk + i] = h[i];
    }
    __syncthreads();
    for (int i = 0; i < kDepth; ++i) {
      float x[4], y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[q] = sa[(threadIdx.x >> 4) + 16 * q][i];
        y[q] = sb[(threadIdx.x & 15) + 16 * q][i];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int p = 0; p < 4; ++p) acc[q][p] = fmaf(x[q], y[p], acc[q][p]);
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int r = (threadIdx.x >> 4) + 16 * q;
      const int64_t n = n0 + (threadIdx.x & 15) + 16 * p;
      if (r < count && n < n_out)
        reinterpret_cast<T*>(d)[(row + r) * n_out + n] = from_float<T>(acc[q][p] * alpha);
    }
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" int fp4_gemm_tn(void* D, int type, const fp4_matrix_t* a, const fp4_matrix_t* b,
                           float alpha, void* stream) {
  bool any_a = false, any_b = false;
  int rc = check_matrix(a, &any_a);
  if (rc != GEMM_OK) return rc;
  if ((rc = check_matrix(b, &any_b)) != GEMM_OK) return rc;
  if (!valid_type(type) || !std::isfinite(alpha) || a->format != b->format || a->cols != b->cols ||
      a->groups != b->groups || b->offsets)
    return GEMM_ERR_INVALID_VALUE;
  const int64_t n_out = b->group_rows;
  if (a->rows == 0 || n_out == 0) return GEMM_OK;
  if (!D) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(D, 2)) return GEMM_ERR_MISALIGNED;
  const uint64_t dbytes = static_cast<uint64_t>(a->rows) * n_out * 2;
  for (const fp4_matrix_t* m : {a, b})
    if (m->cols > 0 && (overlaps(D, dbytes, m->codes, code_bytes(m)) ||
                        overlaps(D, dbytes, m->scales, scale_bytes(m))))
      return GEMM_ERR_INVALID_VALUE;
  int sms = 0;
  if ((rc = require_device(&sms)) != GEMM_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->cols == 0) return write_empty_sum(D, nullptr, 0.0f, a->rows * n_out, sms, s);
  const Fp4View va = view_of(a), vb = view_of(b);
  alpha *= va.up * vb.up;
  const int64_t tiles = a->offsets ? a->rows / kTile + a->groups + 1
                                   : a->groups * ((a->group_rows + kTile - 1) / kTile);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((n_out + kTile - 1) / kTile));
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kThreads), 0, s, static_cast<uint16_t*>(D), va, vb, alpha);
  };
  if (type == MOE_F16)
    return a->format == FP4_NV ? go(fp4_gemm_kernel<__half, FP4_NV>)
                               : go(fp4_gemm_kernel<__half, FP4_MX>);
  return a->format == FP4_NV ? go(fp4_gemm_kernel<__nv_bfloat16, FP4_NV>)
                             : go(fp4_gemm_kernel<__nv_bfloat16, FP4_MX>);
}

extern "C" int fp4_get_device_error(void* stream, uint32_t* raw) {
  const int rc = require_device(nullptr);
  if (rc != GEMM_OK) return rc;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (raw) *raw = 0;
  return GEMM_OK;
}
