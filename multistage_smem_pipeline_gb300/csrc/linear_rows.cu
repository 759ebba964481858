// Rows before the products of linear layers: the gradient of the sums, dz =
// grad_out act'(z), with its sums over rows for the bias; and copies of rows that
// do not start on 16-byte boundaries.
#include "linear_rows.cuh"

namespace gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Elements [e, e + 8) of a row of n that starts at any 2-byte address.
template <bool kAligned>
__device__ __forceinline__ Pack window(const uint16_t* row, int e, int n) {
  return load8<kAligned>(row, e, n);
}

// One block: 256 columns (a lane has eight) of a strip of rows, which its warps take by
// turns, four rows of loads in flight each.  Memory bounds it: reads of grad_out
// and z and the write of dz.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads)
    grad_rows_kernel(const GradRows p) {
  constexpr int kAhead = 4;
  __shared__ float partial[kWarps][256 + 8];
  __shared__ int found[3];   // group, first row, rows
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int strip = blockIdx.y;
  const int n = static_cast<int>(p.grad.cols);
  if (threadIdx.x == 0) found[2] = 0;
  __syncthreads();
  grid_dependency_wait();
  if (p.offsets) {
    // the group whose strips this one is among
    for (int g = threadIdx.x; g < p.groups; g += kThreads) {
      const int first = p.offsets[g], end = p.offsets[g + 1];
      const int at = strip_of(first, g, p.strip_rows);
      if (at <= strip && strip < strip_of(end, g + 1, p.strip_rows)) {
        found[0] = g;
        found[1] = first + (strip - at) * p.strip_rows;
        found[2] = min(p.strip_rows, end - found[1]);   // none: a group's spare strip
      }
    }
  } else if (threadIdx.x == 0) {
    found[1] = strip * p.strip_rows;
    found[2] = min(p.strip_rows, static_cast<int>(p.grad.rows) - found[1]);
  }
  __syncthreads();
  const int rows = found[2];
  if (rows <= 0) return;
  const int64_t row0 = found[1];
  const int c = blockIdx.x * 256 + 8 * lane;
  const bool live = c < n;
  const uint16_t* const grad = static_cast<const uint16_t*>(p.grad.ptr);
  const uint16_t* const z = static_cast<const uint16_t*>(p.preact);
  const int64_t dz_ld = copy_ld(n);
  float sum[8] = {};
  for (int r0 = warp; live && r0 < rows; r0 += kAhead * kWarps) {
    Pack g[kAhead], s[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kWarps;
      if (r < rows) {
        g[i] = window<kAligned>(grad + (row0 + r) * p.grad.ld, c, n);
        if (z) s[i] = window<kAligned>(z + (row0 + r) * n, c, n);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kWarps;
      if (r >= rows) break;
      float v[8];
      unpack<T>(g[i], v);
      if (z) {
        float zs[8];
        unpack<T>(s[i], zs);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= activation_slope(zs[e], p.activation);
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
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col >= n) return;
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    total += partial[w][(threadIdx.x & 7) * 32 + (threadIdx.x >> 3)];
  p.strips[static_cast<int64_t>(strip) * n + col] = total;
}

__global__ void __launch_bounds__(kThreads) copy_rows_kernel(uint16_t* dst, const Rows src) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int n = static_cast<int>(src.cols);
  const int64_t ld = copy_ld(n);
  const int64_t per = ld / 8, total = src.rows * per;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += step) {
    const int64_t r = i / per;
    const int e = static_cast<int>(i - r * per) * 8;
    const uint16_t* const row = static_cast<const uint16_t*>(src.ptr) + r * src.ld;
    *reinterpret_cast<Pack*>(dst + r * ld + e) = window<false>(row, e, n);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sum_strips_kernel(const LinearParams p) {
  extern __shared__ GroupStart start[];
  grid_launch_dependents();
  grid_dependency_wait();
  if (threadIdx.x < 32) linear_starts<kLinM>(p, start, threadIdx.x);
  __syncthreads();
  linear_sum_strips<T>(p, start, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x,
                       static_cast<int64_t>(gridDim.x) * kThreads);
}

}  // namespace

int copy_rows(void* dst, const Rows& src, int sms, cudaStream_t stream) {
  const int64_t pieces = src.rows * (copy_ld(src.cols) / 8);
  const int64_t blocks = std::min<int64_t>((pieces + kThreads - 1) / kThreads, 8LL * sms);
  return launch_pdl(copy_rows_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream,
                    1u, static_cast<uint16_t*>(dst), src);
}

int grad_rows(const GradRows& g, cudaStream_t stream) {
  const bool aligned = loads_as_is(g.grad) && (!g.preact || (aligned_to(g.preact, 16) && g.grad.cols % 8 == 0)) &&
                       g.grad.cols % 8 == 0;
  const int64_t strips = g.offsets ? g.grad.rows / g.strip_rows + g.groups
                                   : (g.grad.rows + g.strip_rows - 1) / g.strip_rows;
  const dim3 grid(static_cast<unsigned>((g.grad.cols + 255) / 256), static_cast<unsigned>(strips));
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, 1u, g);
  };
  if (g.type == MOE_F16)
    return aligned ? go(grad_rows_kernel<__half, true>) : go(grad_rows_kernel<__half, false>);
  return aligned ? go(grad_rows_kernel<__nv_bfloat16, true>)
                 : go(grad_rows_kernel<__nv_bfloat16, false>);
}

int sum_strips(const LinearParams& p, int type, int sms, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(p.groups) * p.m;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((n + kThreads - 1) / kThreads, 8LL * sms)));
  const size_t smem = (p.groups + 1) * sizeof(GroupStart);
  return type == MOE_F16
             ? launch_pdl(sum_strips_kernel<__half>, grid, dim3(kThreads), smem, stream, 1u, p)
             : launch_pdl(sum_strips_kernel<__nv_bfloat16>, grid, dim3(kThreads), smem, stream, 1u, p);
}

}  // namespace gb300
