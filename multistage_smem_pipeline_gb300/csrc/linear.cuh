// What the kernels of linear layers share: the three products and how their
// operands lie, parameters, tiles, waits, and the epilogue.
//
// The products of a layer with weights w (out x in), for the rows of a group:
//   forward  z = x w^T        D rows x out, sums over in
//   grad_x   dz w             D rows x in,  sums over out
//   grad_w   dz^T x           D out x in,   sums over rows
// The tensor cores take D = A B^T, each operand either with the summed index
// contiguous (K-major) or with the other one (MN-major), so nothing is
// transposed in memory:
//              A                      B
//   forward    x       K-major        w        K-major
//   grad_x     dz      K-major        w        MN-major
//   grad_w     dz^T    MN-major       x^T      MN-major
// D's rows are the instruction's M, so that an accumulator lane is a row of D
// and a row's columns lie next to each other for the epilogue.
//
// Groups are ragged in rows: in D's rows for the first two, in the summed index
// for grad_w.  A tile of D ends with its group; the rows of the next group that
// its last box of A brings along end in accumulator lanes that are not stored.
// grad_w has to keep them out of the sums: it stops at the group's last 16 rows
// and zeroes, in shared memory, what of those is not the group's, in both
// operands (a NaN there would come through a zero in the other).  w is a
// tensor of three dimensions, so that boxes past an expert's rows read zeros.
#pragma once
#include <cuda.h>

#include <algorithm>

#include "linear.h"
#include "moe_common.cuh"
#include "tensor_map.cuh"

namespace gb300 {

constexpr int kLinM = 128;            // rows of D per CTA: one accumulator lane each
constexpr int kLinK = 64;             // summed elements of a stage: 128 bytes, a swizzle row
constexpr int kLinEpiWarps = 8;
constexpr int kLinThreads = 64 + 32 * kLinEpiWarps;
constexpr int kLinMaxStages = 12;
constexpr int kLinMaxTile = 256;      // columns of D
constexpr uint32_t kLinABytes = kLinM * kLinK * 2;
constexpr uint32_t kLinChunkBytes = 64 * kLinK * 2;  // MN-major: 64 columns by 64 of the sum
constexpr uint32_t kLinBufBytes = 32 * 32 * 4;       // an epilogue warp's 32 x 32 sums
constexpr uint32_t kLinSmemLimit = 232448;

struct LinearParams {
  uint16_t* out;             // D, rows contiguous
  uint16_t* preact;          // forward: z, or null
  const uint16_t* bias;      // forward: groups x n, or null
  const uint16_t* residual;  // forward: or null
  int64_t ldr;
  const int32_t* offsets;    // of the groups of rows; null: one group
  const float* strips;       // grad_w: sums of dz over strips of rows (linear_rows.cuh), or null
  uint16_t* grad_bias;
  int32_t strip_rows;
  int32_t rows;              // of all groups, and those of none
  int32_t m;                 // grad_w: rows of a group's D
  int32_t n;                 // columns of D
  int32_t k;                 // forward, grad_x: length of the sums
  int32_t groups;
  int32_t tile;              // columns of a tile
  int32_t m_tiles, n_tiles;  // of D; m_tiles: grad_w's, of a group
  int32_t box_rows;          // forward, grad_x: rows that one copy of A loads
  int32_t stages, split;
  int32_t activation;
  int32_t vector;            // D, bias and residual can be accessed 16 bytes at a time
  int32_t inject;            // 1: leave out each CTA's first loads
  int32_t error_word;
  uint64_t timeout_ns;
};

__host__ __device__ constexpr bool a_mn(int product) { return product == LINEAR_GRAD_W; }
__host__ __device__ constexpr bool b_mn(int product) { return product != LINEAR_FORWARD; }

// Shared memory past the ring and the epilogue's buffers: barriers, the tensor
// memory address, the abort flag, and where each group starts; 1 KiB to align.
constexpr uint32_t kLinBars = 3 * kLinMaxStages + 5;
__host__ __device__ constexpr uint32_t linear_fixed_bytes(int groups) {
  return 8 * kLinBars + 24 + 8 * (groups + 1) + 1024;
}

// ------------------------------------------------------------------ PTX
// Instruction descriptor of kind::f16: D fp32 (bits 4-5 = 1), A and B of the
// same type (bits 7-9 and 10-12: 0 fp16, 1 bf16), MN-major A and B (bits 15 and
// 16), N >> 3 in bits 17-22, M >> 4 in bits 24-28.
template <typename T, int kProduct>
__device__ __forceinline__ constexpr uint32_t linear_idesc(int m, int n) {
  return (1u << 4) | (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u) |
         (a_mn(kProduct) ? 1u << 15 : 0u) | (b_mn(kProduct) ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <bool kMn>
__device__ __forceinline__ uint64_t linear_desc(uint32_t smem_addr) {
  return kMn ? sw128_mnmajor_desc(smem_addr, kLinChunkBytes) : sw128_kmajor_desc(smem_addr);
}
// 16 of the sum further, in the descriptor's units of 16 bytes
template <bool kMn>
__device__ __forceinline__ constexpr uint32_t linear_desc_step() { return kMn ? 128u : 2u; }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, uint32_t a, uint32_t b,
                                              uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

// ------------------------------------------------------------------ waits
enum LinearWait : uint32_t { kLinEmpty = 1, kLinFull = 2, kLinTmemEmpty = 3, kLinTmemFull = 4,
                             kLinPeer = 5 };

// The first error of the launches on a given stream (the host maps streams to
// words); 0: none.
__device__ uint32_t g_linear_error[kErrorWords];

// Waits for phase `parity` of `bar`; gives up when the CTA does, or after the
// limit, which it records.  kCluster: for what other CTAs of the cluster wrote.
template <bool kCluster = false>
__device__ __forceinline__ bool linear_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                            uint32_t site, const LinearParams& p) {
  const auto done = [&] {
    return kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  };
  if (done()) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (done()) return true;
    if ((it & 31u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > p.timeout_ns) {
        *abort_flag = 1;
        atomicCAS(&g_linear_error[p.error_word], 0u,
                  static_cast<uint32_t>(GEMM_ERR_TIMEOUT) | (site << 8));
        return false;
      }
    }
  }
}

// The same by a whole warp: it goes on, or gives up, together.
template <bool kCluster = false>
__device__ __forceinline__ bool linear_wait_warp(uint32_t bar, uint32_t parity,
                                                 volatile int* abort_flag, uint32_t site,
                                                 const LinearParams& p) {
  return __all_sync(0xffffffffu, linear_wait<kCluster>(bar, parity, abort_flag, site, p));
}

// A wait on the way out, whether or not the CTA gave up.
__device__ __forceinline__ void linear_wait_drain(uint32_t bar, uint32_t parity,
                                                  uint64_t timeout_ns) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return;
    if ((it & 31u) == 0 && global_timer_ns() - t0 > timeout_ns) return;
  }
}

// ------------------------------------------------------------------ tiles
struct LinearTile {
  int32_t group;
  int32_t row;     // of D: first row (grad_w: within the group's D)
  int32_t count;   // rows of the tile, at most its height
  int32_t col;     // first column
  int32_t k_row;   // grad_w: the first summed row
  int32_t k_len;   // length of the sums
};

// Row tiles that walk over the columns together, so that what runs at once
// shares operands in L2.
constexpr int kLinRaster = 8;

// Row tile and column tile of tile t among m_tiles x n_tiles.
__device__ __forceinline__ void linear_raster(int t, int m_tiles, int n_tiles, int* mt, int* nt) {
  if (m_tiles == 1) {
    *mt = 0;
    *nt = t;
    return;
  }
  const int band = t / (kLinRaster * n_tiles);
  const int in = t - band * kLinRaster * n_tiles;
  const int wide = min(kLinRaster, m_tiles - band * kLinRaster);
  *nt = wide == kLinRaster ? in / kLinRaster : in / wide;
  *mt = band * kLinRaster + in - *nt * wide;
}

// Tiles of all groups.
template <int kProduct>
__device__ __forceinline__ int linear_tiles(const LinearParams& p, const GroupStart* start) {
  return kProduct == LINEAR_GRAD_W ? p.groups * p.m_tiles * p.n_tiles
                                   : start[p.groups].tiles * p.n_tiles;
}

// kHeight: rows of a tile.
template <int kProduct, int kHeight>
__device__ __forceinline__ LinearTile linear_tile(int t, const LinearParams& p,
                                                  const GroupStart* start) {
  LinearTile o;
  int mt, nt;
  if (kProduct == LINEAR_GRAD_W) {
    const int per = p.m_tiles * p.n_tiles;
    o.group = p.groups > 1 ? t / per : 0;
    linear_raster(t - o.group * per, p.m_tiles, p.n_tiles, &mt, &nt);
    o.row = mt * kHeight;
    o.count = min(kHeight, p.m - o.row);
    o.k_row = start[o.group].row;
    o.k_len = start[o.group + 1].row - o.k_row;
  } else {
    int lo = 0, hi = p.groups - 1;  // the last group with tiles * n_tiles <= t before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid].tiles * p.n_tiles <= t) lo = mid;
      else hi = mid - 1;
    }
    const int first = start[lo].row, rows = start[lo + 1].row - first;
    linear_raster(t - start[lo].tiles * p.n_tiles, (rows + kHeight - 1) / kHeight, p.n_tiles, &mt,
                  &nt);
    o.group = lo;
    o.row = first + mt * kHeight;
    o.count = min(kHeight, rows - mt * kHeight);
    o.k_row = 0;
    o.k_len = p.k;
  }
  o.col = nt * p.tile;
  return o;
}

// Where each group starts, by one warp.
template <int kHeight>
__device__ __forceinline__ void linear_starts(const LinearParams& p, GroupStart* start, int lane) {
  if (p.offsets) {
    find_groups<kHeight>(p.offsets, p.groups, start, lane);
  } else {  // one group, or none of any rows
    for (int g = lane; g <= p.groups; g += 32)
      start[g] = g ? GroupStart{(p.rows + kHeight - 1) / kHeight, p.rows} : GroupStart{0, 0};
  }
}

// Whether there is anything to sum, and the tensor maps mean something.
template <int kProduct>
__device__ __forceinline__ bool linear_has_sums(const LinearParams& p) {
  return kProduct == LINEAR_GRAD_W ? p.rows > 0 : p.k > 0;
}

// Stage kb's steps of 16 along the sum.
__device__ __forceinline__ int linear_steps(const LinearTile& t, int kb) {
  return min(kLinK / 16, (t.k_len - kb * kLinK + 15) >> 4);
}
// grad_w: whether the sum ends inside a step, so that rows of the next group (or
// of none) are in it.  (Past the last row of all the copies bring zeros.)
__device__ __forceinline__ bool linear_ragged(const LinearTile& t, int kb, const LinearParams& p) {
  return p.offsets && (t.k_len & 15) && t.k_len - kb * kLinK < kLinK;
}

// Zeroes, in `chunks` chunks of 64 columns, the rows of the stage's last step that
// are past the sum's end.  By a warp; the MMAs see it after the proxy fence.
__device__ __forceinline__ void linear_zero_rows(uint32_t at, int chunks, int valid, int lane) {
  const int pieces = (((valid + 15) & ~15) - valid) * 8;
  for (int c = 0; c < chunks; ++c)
    for (int i = lane; i < pieces; i += 32)
      st_shared_v4(at + c * kLinChunkBytes + valid * 128u + i * 16u, 0, 0, 0, 0);
}

// ------------------------------------------------------------------ epilogue
// 1 / (1 + e^-u) and 1 / (1 + e^u), with their relative accuracy on both sides: the
// exponential is at most 1, the denominator between 1 and 2.
struct Sigmoids {
  float up, down;
};
__device__ __forceinline__ Sigmoids sigmoids(float u) {
  const float e = __expf(-fabsf(u)), r = __fdividef(1.0f, 1.0f + e), s = e * r;
  return u < 0.0f ? Sigmoids{s, r} : Sigmoids{r, s};
}

// (1 + tanh u) / 2 is the sigmoid of 2u; 1.5957691 = 2 sqrt(2 / pi).
__device__ __forceinline__ float gelu_tanh_argument(float z) {
  return 1.5957691f * z * fmaf(0.044715f, z * z, 1.0f);
}

__device__ __forceinline__ float activate(float z, int activation) {
  switch (activation) {
    case LINEAR_RELU:
      return z < 0.0f ? 0.0f : z;  // a NaN stays
    case LINEAR_GELU:
      return 0.5f * z * erfcf(z * -0.70710678f);  // erfc: no cancellation far below 0
    case LINEAR_GELU_TANH:
      return z * sigmoids(gelu_tanh_argument(z)).up;
    case LINEAR_SILU:
      return z * sigmoids(z).up;
    default:
      return z;
  }
}

// act'(z).  Past 100 it is 0 or 1 in fp32, and products of what overflows and what
// vanishes there would be NaN.
__device__ __forceinline__ float activation_slope(float z, int activation) {
  if (fabsf(z) > 100.0f) z = copysignf(100.0f, z);
  switch (activation) {
    case LINEAR_RELU:
      return z > 0.0f ? 1.0f : 0.0f;
    case LINEAR_GELU:
      return fmaf(z * 0.39894228f, __expf(-0.5f * z * z), 0.5f * erfcf(z * -0.70710678f));
    case LINEAR_GELU_TANH: {
      const Sigmoids s = sigmoids(gelu_tanh_argument(z));
      return fmaf(z * fmaf(0.21406445f, z * z, 1.5957691f), s.up * s.down, s.up);
    }
    case LINEAR_SILU: {
      const Sigmoids s = sigmoids(z);
      return s.up * fmaf(z, s.down, 1.0f);
    }
    default:
      return 1.0f;
  }
}

// An epilogue warp's 32 x 32 sums pass through shared memory from the layout of
// the accumulator (a lane is a row) to that of memory (four lanes are a row's 32
// columns, eight of them each), so that bias, residual, z and D are read and
// written 16 bytes a lane, 64 bytes of a row at once.  Piece j (of 16 bytes) of row r
// is at j ^ (r & 7): neither side has bank conflicts.
__device__ __forceinline__ uint32_t linear_piece(uint32_t buf, int row, int piece) {
  return buf + row * 128u + (static_cast<uint32_t>(piece ^ (row & 7)) << 4);
}

// 32 columns of a warp's 32 rows from the accumulator; zeros where nothing was summed
// (`any`).  The load and the wait for it are one statement: until the wait its registers
// are still being written, and the compiler, which does not know that, would move
// what it found in them, or use them for something else, in between.
__device__ __forceinline__ void linear_sums(uint32_t taddr, bool any, uint32_t (&r)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = any ? r[i] : 0u;
}

__device__ __forceinline__ void linear_put_row(uint32_t buf, int lane, const uint32_t (&r)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    st_shared_v4(linear_piece(buf, lane, j), r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
}

// What a chunk's epilogue reads from memory, asked for before its sums are there.
struct LinearExtras {
  Pack bias;
  Pack residual[4];
};

template <int kProduct>
__device__ __forceinline__ LinearExtras linear_extras(const LinearParams& p, int group, int64_t row,
                                                      int live, int col, int lane) {
  LinearExtras x = {};
  if (kProduct != LINEAR_FORWARD || !p.vector) return x;
  const int c = col + 8 * (lane & 3);
  if (c >= p.n) return x;
  if (p.bias)
    x.bias = *reinterpret_cast<const Pack*>(p.bias + static_cast<int64_t>(group) * p.n + c);
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      if (r < live)
        x.residual[i] = *reinterpret_cast<const Pack*>(p.residual + (row + r) * p.ldr + c);
    }
  }
  return x;
}

// The chunk whose first row of D is `row` and first column `col`; `live` of its rows are
// the tile's.  Its sums are those of `parts` buffers `part_bytes` apart, added in order.
template <typename T, int kProduct>
__device__ __forceinline__ void linear_finish(uint32_t buf, int parts, uint32_t part_bytes,
                                              const LinearParams& p, LinearExtras& x, int group,
                                              int64_t row, int live, int col, int lane) {
  constexpr bool kForward = kProduct == LINEAR_FORWARD;
  if (p.vector) {
    const int c = col + 8 * (lane & 3);
    float bias[8];
    if (kForward) unpack<T>(x.bias, bias);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      if (8 * i >= live) break;
      const int r = 8 * i + (lane >> 2);
      float v[8] = {};
      for (int s = 0; s < parts; ++s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 q = ld_shared_v4(linear_piece(buf + s * part_bytes, r, 2 * (lane & 3) + h));
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * h + e] += __uint_as_float(w[e]);
        }
      }
      if (r < live && c < p.n) {
        const int64_t at = (row + r) * p.n + c;
        if (kForward) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += bias[e];
          if (p.preact) *reinterpret_cast<Pack*>(p.preact + at) = pack<T>(v);
          if (p.activation != LINEAR_NONE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = activate(v[e], p.activation);
          }
          if (p.residual) {
            float res[8];
            unpack<T>(x.residual[0], res);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += res[e];
          }
        }
        *reinterpret_cast<Pack*>(p.out + at) = pack<T>(v);
      }
      if (kForward) {
#pragma unroll
        for (int e = 0; e < 3; ++e) x.residual[e] = x.residual[e + 1];
      }
    }
    return;
  }
  // Rows that are not aligned: a lane is a column, a row at a time.
  const int c = col + lane;
  if (c >= p.n) return;
  const float bias = kForward && p.bias
                         ? to_float(reinterpret_cast<const T*>(p.bias)[static_cast<int64_t>(group) * p.n + c])
                         : 0.0f;
#pragma unroll 1
  for (int r0 = 0; r0 < live; r0 += 8) {
    T res[8] = {};
    if (kForward && p.residual) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r0 + i < live)
          res[i] = reinterpret_cast<const T*>(p.residual)[(row + r0 + i) * p.ldr + c];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + i;
      float v = 0.0f;
      for (int s = 0; s < parts; ++s) {
        float part;
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(part)
                     : "r"(linear_piece(buf + s * part_bytes, r, lane >> 2) + 4u * (lane & 3))
                     : "memory");
        v += part;
      }
      if (r >= live) continue;
      const int64_t at = (row + r) * p.n + c;
      if (kForward) {
        v += bias;
        if (p.preact) reinterpret_cast<T*>(p.preact)[at] = from_float<T>(v);
        v = activate(v, p.activation);
        if (p.residual) v += to_float(res[i]);
      }
      reinterpret_cast<T*>(p.out)[at] = from_float<T>(v);
    }
  }
}

// ------------------------------------------------------------------ grad_bias
// The sums of dz over strips of strip_rows rows (the last of a group is shorter) are
// rows of `strips`, those of group g from offsets[g] / strip_rows + g on: no group
// needs to know how many strips others have.
__host__ __device__ __forceinline__ int strip_of(int row, int group, int strip_rows) {
  return row / strip_rows + group;
}

// grad_bias from the strips, added in their order, by threads first, first + step ...
// of the grid.  In the products' kernels: by the epilogue's, which wait for the
// first sums anyway.
template <typename T>
__device__ __forceinline__ void linear_sum_strips(const LinearParams& p, const GroupStart* start,
                                                  int64_t first, int64_t step) {
  const int64_t n = static_cast<int64_t>(p.groups) * p.m;
  for (int64_t i = first; i < n; i += step) {
    const int g = static_cast<int>(i / p.m), row = start[g].row;
    const int count = (start[g + 1].row - row + p.strip_rows - 1) / p.strip_rows;
    const float* at =
        p.strips + static_cast<int64_t>(strip_of(row, g, p.strip_rows)) * p.m + (i - static_cast<int64_t>(g) * p.m);
    float sum = 0.0f;
    int s = 0;
    for (; s + 8 <= count; s += 8) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = at[static_cast<int64_t>(s + e) * p.m];
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[e];
    }
    for (; s < count; ++s) sum += at[static_cast<int64_t>(s) * p.m];
    reinterpret_cast<T*>(p.grad_bias)[i] = from_float<T>(sum);
  }
}

template <typename T>
__device__ __forceinline__ void linear_sum_strips(const LinearParams& p, const GroupStart* start) {
  if (!p.strips) return;
  linear_sum_strips<T>(p, start,
                       static_cast<int64_t>(blockIdx.x) * (32 * kLinEpiWarps) + threadIdx.x - 64,
                       static_cast<int64_t>(gridDim.x) * (32 * kLinEpiWarps));
}

// First row of a tile's part of D in memory.
template <int kProduct>
__device__ __forceinline__ int64_t linear_out_row(const LinearTile& t, const LinearParams& p) {
  return kProduct == LINEAR_GRAD_W ? static_cast<int64_t>(t.group) * p.m + t.row
                                   : static_cast<int64_t>(t.row);
}

// Rows of no group are zero, by every epilogue thread of the grid.
template <int kProduct>
__device__ __forceinline__ void linear_zero_tail(const LinearParams& p, const GroupStart* start) {
  if (kProduct == LINEAR_GRAD_W || !p.offsets) return;
  const int64_t from = static_cast<int64_t>(start[p.groups].row) * p.n;
  const int64_t end = static_cast<int64_t>(p.rows) * p.n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (32 * kLinEpiWarps);
  for (int64_t i = from + static_cast<int64_t>(blockIdx.x) * (32 * kLinEpiWarps) + threadIdx.x - 64;
       i < end; i += step) {
    p.out[i] = 0;
    if (kProduct == LINEAR_FORWARD && p.preact) p.preact[i] = 0;
  }
}

}  // namespace gb300
