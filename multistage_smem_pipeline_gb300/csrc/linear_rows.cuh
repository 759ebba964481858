// What linear layers do with rows before their products (linear_rows.cu).
#pragma once
#include "linear.cuh"

namespace gb300 {

// Rows of `cols` elements, `ld` apart.
struct Rows {
  const void* ptr;
  int64_t rows, cols, ld;
};

// The kernels' tensor maps take these rows as they are.
inline bool loads_as_is(const Rows& r) { return aligned_to(r.ptr, 16) && r.ld % 8 == 0; }
// Elements between the rows of a copy that they can take.
__host__ __device__ inline int64_t copy_ld(int64_t cols) { return (cols + 7) / 8 * 8; }

// Rows of a strip for rows x cols: 32, more where there are blocks enough (of 256 columns
// each) to fill the GPU's SMs twice over.
inline int strip_rows_for(int64_t rows, int64_t cols) {
  int64_t s = 32;
  while (rows / (2 * s) * ((cols + 255) / 256) >= 1216 || rows / s > 4096) s *= 2;
  return static_cast<int>(s);
}

// What a call has to do with rows before its products, in one launch.
struct PrepareRows {
  // dz = grad_out act'(preact), for the rows that are in a group
  Rows grad;                 // grad_out; no rows: nothing of this
  const void* preact;        // contiguous; null for LINEAR_NONE
  void* dz;                  // copy_ld(cols) between rows; or null
  float* strips;             // sums of dz over strips of rows; or null
  const int32_t* offsets;    // or null: one group
  int groups, strip_rows, type, activation;
  // copies, copy_ld(cols) between rows, 16-byte aligned; null: none
  Rows from[2];
  void* to[2];
};
int prepare_rows(const PrepareRows& p, cudaStream_t stream);

// grad_bias from the strips alone (else a product's kernel does that).
int sum_strips(const LinearParams& p, int type, int sms, cudaStream_t stream);

}  // namespace gb300
