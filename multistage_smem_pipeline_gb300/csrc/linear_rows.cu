// Rows before the products of linear layers: the gradient of the sums, dz =
// grad_out act'(z), with its sums over rows for the bias; and copies of rows that
// do not start on 16-byte boundaries.
//
// dz is bound by memory: read and written once, 8192 x 4096 gelu in 35.5 us (5.7 TB/s) and 64
// groups of 32768 x 2048 silu in 66 (6.1), without the sum of the strips.
#include "linear_rows.cuh"

namespace gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

constexpr int kCopyAhead = 4;
constexpr int kCopyPieces = kCopyAhead * kThreads;  // of 16 bytes, that a block copies

// Blocks of a launch: first those of dz, then those of each copy.
struct PrepareParams {
  PrepareRows p;
  int col_blocks;            // of dz: 256 columns each
  int64_t first_copy[2];     // block
};

__device__ void copy_block(const Rows& src, uint16_t* dst, int64_t block) {
  const int n = static_cast<int>(src.cols);
  const int64_t ld = copy_ld(n);
  const uint32_t per = static_cast<uint32_t>(ld / 8);
  const int64_t row0 = block * kCopyPieces / per;
  const uint32_t piece0 = static_cast<uint32_t>(block * kCopyPieces - row0 * per);
  Pack v[kCopyAhead];
  int64_t row[kCopyAhead];
  int e[kCopyAhead];
#pragma unroll
  for (int i = 0; i < kCopyAhead; ++i) {
    const uint32_t at = piece0 + threadIdx.x + i * kThreads;
    row[i] = row0 + at / per;
    e[i] = static_cast<int>(at % per) * 8;
    if (row[i] < src.rows)
      v[i] = load8<false>(static_cast<const uint16_t*>(src.ptr) + row[i] * src.ld, e[i], n);
  }
#pragma unroll
  for (int i = 0; i < kCopyAhead; ++i)
    if (row[i] < src.rows) *reinterpret_cast<Pack*>(dst + row[i] * ld + e[i]) = v[i];
}

// A block of dz: 256 columns (a lane has eight) of a strip of rows, which its warps
// take by turns, two rows of loads in flight each.  Memory bounds it: reads of
// grad_out and z and the write of dz.
template <typename T, bool kAligned, int kActivation>
__global__ void __launch_bounds__(kThreads, 4)
    prepare_kernel(const __grid_constant__ PrepareParams q) {
  constexpr int kAhead = 2;
  constexpr bool kSlope = kActivation != LINEAR_NONE;
  __shared__ float partial[kWarps][256 + 8];
  __shared__ int found[2];   // first row, rows
  const PrepareRows& p = q.p;
  if (threadIdx.x == 0) {
    grid_launch_dependents();
    found[1] = 0;
  }
  grid_dependency_wait();
  const int64_t block = blockIdx.x;
  if (block >= q.first_copy[0]) {
    const int which = block >= q.first_copy[1];
    copy_block(p.from[which], static_cast<uint16_t*>(p.to[which]), block - q.first_copy[which]);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int strip = static_cast<int>(block / q.col_blocks);
  const int col0 = static_cast<int>(block - static_cast<int64_t>(strip) * q.col_blocks) * 256;
  const int n = static_cast<int>(p.grad.cols);
  int64_t row0;
  int rows;
  if (p.offsets) {
    // the group whose strips this one is among
    __syncthreads();
    for (int g = threadIdx.x; g < p.groups; g += kThreads) {
      const int first = p.offsets[g], end = p.offsets[g + 1];
      const int at = strip_of(first, g, p.strip_rows);
      if (at <= strip && strip < strip_of(end, g + 1, p.strip_rows)) {
        found[0] = first + (strip - at) * p.strip_rows;
        found[1] = min(p.strip_rows, end - found[0]);   // none: a group's spare strip
      }
    }
    __syncthreads();
    row0 = found[0];
    rows = found[1];
  } else {
    row0 = static_cast<int64_t>(strip) * p.strip_rows;
    rows = static_cast<int>(min(static_cast<int64_t>(p.strip_rows), p.grad.rows - row0));
  }
  if (rows <= 0) return;
  const int c = col0 + 8 * lane;
  const uint16_t* const grad = static_cast<const uint16_t*>(p.grad.ptr);
  const uint16_t* const z = static_cast<const uint16_t*>(p.preact);
  const int64_t dz_ld = copy_ld(n);
  float sum[8] = {};
  for (int r0 = warp; c < n && r0 < rows; r0 += kAhead * kWarps) {
    Pack g[kAhead], s[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kWarps;
      if (r < rows) {
        g[i] = load8<kAligned>(grad + (row0 + r) * p.grad.ld, c, n);
        if (kSlope) s[i] = load8<kAligned>(z + (row0 + r) * n, c, n);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kWarps;
      if (r >= rows) break;
      float v[8];
      unpack<T>(g[i], v);
      if (kSlope) {
        float zs[8];
        unpack<T>(s[i], zs);
#pragma unroll
        for (int e = 0; e < 8; ++e)  // rounded, also where nothing but the sum takes it
          v[e] = __fmul_rn(v[e], activation_slope<kActivation>(zs[e]));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[e];
      if (p.dz)
        *reinterpret_cast<Pack*>(static_cast<uint16_t*>(p.dz) + (row0 + r) * dz_ld + c) =
            pack<T>(v);
    }
  }
  if (!p.strips) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) partial[warp][e * 32 + lane] = sum[e];
  __syncthreads();
  const int col = col0 + threadIdx.x;
  if (col >= n) return;
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    total += partial[w][(threadIdx.x & 7) * 32 + (threadIdx.x >> 3)];
  p.strips[strip * strip_ld(n) + col] = total;
}

template <typename T, bool kAligned>
int launch_prepare(const PrepareParams& q, unsigned blocks, cudaStream_t s) {
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, s, 1u, q);
  };
  switch (q.p.activation) {
    case LINEAR_RELU: return go(prepare_kernel<T, kAligned, LINEAR_RELU>);
    case LINEAR_GELU: return go(prepare_kernel<T, kAligned, LINEAR_GELU>);
    case LINEAR_GELU_TANH: return go(prepare_kernel<T, kAligned, LINEAR_GELU_TANH>);
    case LINEAR_SILU: return go(prepare_kernel<T, kAligned, LINEAR_SILU>);
    default: return go(prepare_kernel<T, kAligned, LINEAR_NONE>);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sum_strips_kernel(const LinearParams p) {
  extern __shared__ GroupStart start[];
  grid_launch_dependents();
  grid_dependency_wait();
  if (threadIdx.x < 32) linear_starts(p, start, threadIdx.x);
  __syncthreads();
  linear_sum_strips<T>(p, start, static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5),
                       static_cast<int64_t>(gridDim.x) * kWarps, threadIdx.x & 31);
}

}  // namespace

int prepare_rows(const PrepareRows& p, cudaStream_t stream) {
  PrepareParams q;
  q.p = p;
  q.col_blocks = static_cast<int>((p.grad.cols + 255) / 256);
  const int64_t strips = p.offsets ? p.grad.rows / p.strip_rows + p.groups
                                   : (p.grad.rows + p.strip_rows - 1) / std::max(p.strip_rows, 1);
  int64_t blocks = p.grad.rows > 0 ? q.col_blocks * strips : 0;
  for (int i = 0; i < 2; ++i) {
    q.first_copy[i] = blocks;
    if (p.to[i])
      blocks += (p.from[i].rows * (copy_ld(p.from[i].cols) / 8) + kCopyPieces - 1) / kCopyPieces;
  }
  if (blocks == 0) return GEMM_OK;
  if (blocks > INT_MAX) return GEMM_ERR_INVALID_VALUE;
  const bool aligned = loads_as_is(p.grad) && p.grad.cols % 8 == 0 && aligned_to(p.preact, 16);
  const unsigned n = static_cast<unsigned>(blocks);
  if (p.type == MOE_F16)
    return aligned ? launch_prepare<__half, true>(q, n, stream)
                   : launch_prepare<__half, false>(q, n, stream);
  return aligned ? launch_prepare<__nv_bfloat16, true>(q, n, stream)
                 : launch_prepare<__nv_bfloat16, false>(q, n, stream);
}

int sum_strips(const LinearParams& p, int type, int sms, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(p.groups) * ((p.m + 31) / 32);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((units + kWarps - 1) / kWarps, 8LL * sms)));
  const size_t smem = (p.groups + 1) * sizeof(GroupStart);
  return type == MOE_F16
             ? launch_pdl(sum_strips_kernel<__half>, grid, dim3(kThreads), smem, stream, 1u, p)
             : launch_pdl(sum_strips_kernel<__nv_bfloat16>, grid, dim3(kThreads), smem, stream, 1u, p);
}

}  // namespace gb300
