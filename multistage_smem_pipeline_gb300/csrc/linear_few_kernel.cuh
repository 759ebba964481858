// The forward product for a few rows, without the tensor cores: out[r][n] for up to kRows
// rows of a group at a time.
//
// On the tensor cores the issue loop takes about 356 cycles for a stage, 16 KiB of weights,
// however few the rows are, and tiles of 128 outputs are too few to fill the SMs
// (1 x 4096 x 4096: 32 tiles, 11.6 us; 7.5 so).  Here a warp has four outputs, whose
// weights it reads 16 bytes a lane along the sum; a lane's products go to 4 x kRows
// sums in registers, which the warp's lanes add up at the end, halving the number of
// sums as they halve the distance.  What bounds it is memory (1 x 14336 x 4096: 21.1 us,
// 5.6 TB/s), and for 8 rows the multiplications (35).  `split` warps share a sum where outputs
// are few, and add their parts in order.  x comes from the first-level cache, and is used for four
// outputs at a time.  Rows may start at any 2-byte address: nothing is copied first.
#pragma once
#include "linear.cuh"

namespace gb300 {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewOuts = 4;  // outputs of a warp
// Blocks an SM: with fewer registers each, memory has more asked of it (1 x 14336 x 4096: 21.7
// us by four, 24.5 by two with the next weights already on their way).
__host__ __device__ constexpr int few_blocks(int rows, bool aligned) {
  return rows == 8 ? 2 : rows > 1 || !aligned ? 3 : 4;
}

struct FewParams {
  const uint16_t* x;
  const uint16_t* w;
  int64_t ldx, ldw;
};

// sum += <a, b>, eight products, exact, each added in fp32.
template <typename T>
__device__ __forceinline__ float dot8(const Pack& a, const Pack& b, float sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (std::is_same<T, __half>::value)
      asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %1;\n\tmov.b32 {bl, bh}, %2;\n\t"
          "fma.rn.f32.f16 %0, al, bl, %0;\n\tfma.rn.f32.f16 %0, ah, bh, %0;\n\t}"
          : "+f"(sum)
          : "r"(a.w[i]), "r"(b.w[i]));
    else
      asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %1;\n\tmov.b32 {bl, bh}, %2;\n\t"
          "fma.rn.f32.bf16 %0, al, bl, %0;\n\tfma.rn.f32.bf16 %0, ah, bh, %0;\n\t}"
          : "+f"(sum)
          : "r"(a.w[i]), "r"(b.w[i]));
  }
  return sum;
}

// Elements [e, e + 8) of a row of n, zeros outside it.
template <bool kAligned>
__device__ __forceinline__ Pack load8_clipped(const uint16_t* row, int e, int n) {
  Pack p = load8<kAligned>(row, e, n);
  if (!kAligned && e + 8 > n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e + 2 * i + 1 >= n) p.w[i] &= 0xffffu;
      if (e + 2 * i >= n) p.w[i] = 0;
    }
  }
  return p;
}

// The sums of a warp's lanes, each lane ending with sums of its own in v[0]: while there
// is more than one, a lane keeps half of them.
template <int kN, int kD, int kSize>
__device__ __forceinline__ void add_lanes(float (&v)[kSize], int lane) {
  if constexpr (kD >= 1) {
    if constexpr (kN > 1) {
      const bool upper = lane & kD;
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        const float keep = upper ? v[i + kN / 2] : v[i];
        const float give = upper ? v[i] : v[i + kN / 2];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, kD);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], kD);
    }
    add_lanes<(kN > 1 ? kN / 2 : 1), kD / 2>(v, lane);
  }
}

template <typename T, int kRows, bool kAligned>
__global__ void __launch_bounds__(kFewThreads, few_blocks(kRows, kAligned))
    linear_few(const FewParams f, const LinearParams p) {
  constexpr int kOuts = kFewOuts;
  constexpr int kSums = kOuts * kRows;
  __shared__ float parts[kFewWarps][kSums];
  if (threadIdx.x == 0) grid_launch_dependents();
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp / p.split, part = warp - team * p.split;
  const int per_group = (p.n + kOuts - 1) / kOuts;
  const int unit = static_cast<int>(blockIdx.x) * (kFewWarps / p.split) + team;
  int group = unit / per_group;
  const int n0 = (unit - group * per_group) * kOuts;
  int row = 0, end = group < p.groups ? p.rows : 0;
  if (p.offsets && kRows == 1) {
    // a row, whose group its warps find: most groups have none
    row = group;
    int before = 0;  // groups that end at the row or before it
    for (int g = lane; g < p.groups; g += 32) before += p.offsets[g + 1] <= row;
    group = min(__reduce_add_sync(0xffffffffu, before), p.groups - 1);
    end = min(row + 1, p.offsets[p.groups]);
  } else if (p.offsets && group < p.groups) {
    row = p.offsets[group];
    end = p.offsets[group + 1];
  }
  const uint16_t* const w0 = f.w + (static_cast<int64_t>(group) * p.n + n0) * f.ldw;
  const int outs = min(kOuts, p.n - n0);
  // every team of a block goes round as often as the one with the most rows
  for (; __syncthreads_or(row < end); row += kRows) {
    float sum[kSums] = {};
    if (row < end) {
      const uint16_t* const x0 = f.x + static_cast<int64_t>(row) * f.ldx;
      const int rows = min(kRows, end - row);
      const int step = p.split * 256;
      for (int k = (part * 32 + lane) * 8; k < p.k; k += step) {
        Pack w[kOuts], x[kRows];
#pragma unroll
        for (int o = 0; o < kOuts; ++o)  // past the last output: the first one's again
          w[o] = load8_clipped<kAligned>(w0 + (o < outs ? o : 0) * f.ldw, k, p.k);
#pragma unroll
        for (int r = 0; r < kRows; ++r)  // past the last row: the first one's again
          x[r] = load8_clipped<kAligned>(x0 + (r < rows ? r : 0) * f.ldx, k, p.k);
#pragma unroll
        for (int o = 0; o < kOuts; ++o)
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            sum[o * kRows + r] = dot8<T>(w[o], x[r], sum[o * kRows + r]);
      }
    }
    add_lanes<kSums, 16>(sum, lane);
    constexpr int kSpread = kSums < 32 ? 32 / kSums : 1;  // lanes that end with the same sum
    const int mine = lane / kSpread;                      // the sum that this lane has
    const bool first = lane % kSpread == 0;
    float v = sum[0];
    if (p.split > 1) {
      if (first) parts[warp][mine] = v;
      __syncthreads();
      if (part == 0) {
        v = 0.0f;
        for (int s = 0; s < p.split; ++s) v += parts[warp + s][mine];
      }
    }
    const int n_out = n0 + mine / kRows, r = row + mine % kRows;
    if (row < end && part == 0 && first && n_out < p.n && r < end) {
      const int64_t at = static_cast<int64_t>(r) * p.n + n_out;
      if (p.bias)
        v += to_float(
            reinterpret_cast<const T*>(p.bias)[static_cast<int64_t>(group) * p.n + n_out]);
      if (p.preact) reinterpret_cast<T*>(p.preact)[at] = from_float<T>(v);
      float a[1] = {v};
      activate_all(a, p.activation);
      if (p.residual)
        a[0] += to_float(reinterpret_cast<const T*>(p.residual)[r * p.ldr + n_out]);
      reinterpret_cast<T*>(p.out)[at] = from_float<T>(a[0]);
    }
  }
  if (p.offsets) {  // rows of no group are zero
    const int64_t stop = static_cast<int64_t>(p.rows) * p.n;
    for (int64_t i = static_cast<int64_t>(p.offsets[p.groups]) * p.n +
                     static_cast<int64_t>(blockIdx.x) * kFewThreads + threadIdx.x;
         i < stop; i += static_cast<int64_t>(gridDim.x) * kFewThreads) {
      p.out[i] = 0;
      if (p.preact) p.preact[i] = 0;
    }
  }
}

}  // namespace gb300
