// The 4-bit formats and the layout of their codes and scales (see moe_fp4.h).
#pragma once
#include <algorithm>

#include "moe_common.cuh"

namespace gb300 {

constexpr int kTileRows = 128;    // rows of a scale tile
constexpr int kStageCols = 256;   // columns are padded to this for the scales
constexpr int kChunkBytes = 512;  // 128 rows x 4 blocks

__host__ __device__ constexpr int block_size(int format) { return format == FP4_NV ? 16 : 32; }
// 512-byte chunks of one tile per 256 columns
__host__ __device__ constexpr int chunks_per_stage(int format) { return format == FP4_NV ? 4 : 2; }

__host__ __device__ __forceinline__ int64_t code_pitch(int64_t cols) { return (cols + 31) / 32 * 16; }
__host__ __device__ __forceinline__ int64_t col_stages(int64_t cols) {
  return (cols + kStageCols - 1) / kStageCols;
}

// What a kernel needs to find a matrix's rows and tiles.
struct Fp4View {
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, cols, pitch;
  int64_t tile_bytes;      // of scales
  int64_t group_rows;      // uniform groups
  const int32_t* offsets;  // or null
  int32_t groups;
  float up, down;          // 2^exponent and its inverse
};

// Tiles that a matrix's scales have room for.  By offsets: group g starts at
// tile offsets[g] / 128 + g, and needs ceil(count / 128) of them, which the
// next group's start always leaves: floor((o + c) / 128) - floor(o / 128) + 1
// >= ceil(c / 128).  No sum over the groups is needed to find a tile.
inline int64_t tile_count(int64_t rows, int64_t groups, bool by_offsets) {
  if (by_offsets) return rows / kTileRows + groups;
  return groups * ((rows / groups + kTileRows - 1) / kTileRows);
}

inline int check_format(int format) {
  return format == FP4_NV || format == FP4_MX ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

inline bool fits(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= INT_MAX && cols <= FP4_MAX_COLS;
}

// Checks a matrix's fields; `any` is false where it holds nothing, so that its
// pointers are not looked at.
inline int check_matrix(const fp4_matrix_t* m, bool* any) {
  if (!m || !fits(m->rows, m->cols) || check_format(m->format) != GEMM_OK || m->groups < 1 ||
      m->reserved != 0)
    return GEMM_ERR_INVALID_VALUE;
  if (m->format == FP4_MX ? m->exponent != 0 : (m->exponent < -100 || m->exponent > 100))
    return GEMM_ERR_INVALID_VALUE;
  if (m->offsets) {
    if (m->groups > MOE_MAX_EXPERTS) return GEMM_ERR_INVALID_VALUE;
    if (!aligned_to(m->offsets, 4)) return GEMM_ERR_MISALIGNED;
  } else if (m->group_rows < 0 || m->group_rows > INT_MAX ||
             m->group_rows * m->groups != m->rows) {
    return GEMM_ERR_INVALID_VALUE;
  }
  *any = m->rows > 0 && m->cols > 0;
  if (!*any) return GEMM_OK;
  if (!m->codes || !m->scales) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(m->codes, 16) || !aligned_to(m->scales, 16)) return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}

inline uint64_t code_bytes(const fp4_matrix_t* m) {
  return static_cast<uint64_t>(m->rows) * code_pitch(m->cols);
}

inline uint64_t tile_bytes(int64_t cols, int format) {
  return static_cast<uint64_t>(col_stages(cols)) * chunks_per_stage(format) * kChunkBytes;
}

inline uint64_t scale_bytes(const fp4_matrix_t* m) {
  return static_cast<uint64_t>(tile_count(m->rows, m->groups, m->offsets != nullptr)) *
         tile_bytes(m->cols, m->format);
}

inline uint64_t offset_bytes(const fp4_matrix_t* m) {
  return (static_cast<uint64_t>(m->groups) + 1) * sizeof(int32_t);
}

inline float power_of_two(int e) {  // |e| <= 126
  const uint32_t bits = static_cast<uint32_t>(e + 127) << 23;
  float f;
  std::memcpy(&f, &bits, 4);
  return f;
}

inline Fp4View view_of(const fp4_matrix_t* m) {
  Fp4View v;
  v.codes = static_cast<uint8_t*>(m->codes);
  v.scales = static_cast<uint8_t*>(m->scales);
  v.rows = m->rows;
  v.cols = m->cols;
  v.pitch = code_pitch(m->cols);
  v.tile_bytes = static_cast<int64_t>(tile_bytes(m->cols, m->format));
  v.group_rows = m->group_rows;
  v.offsets = m->offsets;
  v.groups = m->groups;
  v.up = power_of_two(m->exponent);
  v.down = power_of_two(-m->exponent);
  return v;
}

// ------------------------------------------------------------------ device
// Byte of block `b` (counted along the row) of row r (within the tile).
__device__ __forceinline__ int scale_at(int r, int b) {
  return (b >> 2) * kChunkBytes + (r & 31) * 16 + (r >> 5) * 4 + (b & 3);
}

// Rows [row, row + count) and the scale tile of one 128-row tile of a matrix.
// Tile numbers run over the tiles that tile_count() counts and, by offsets,
// one more: those past the last group stand for the rows in no group, with
// tile = -1.
struct TileRows {
  int32_t row, count, tile;
};

// The last g in [0, groups] with offsets[g] / unit + g <= q.
__device__ __forceinline__ int find_group(const int32_t* offsets, int groups, int unit, int64_t q) {
  int lo = 0, hi = groups;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] / unit + mid <= q) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The group of a row below offsets[groups]: the last one that starts at or
// before it (those before that start there too are empty).
__device__ __forceinline__ int group_of_row(const int32_t* offsets, int groups, int32_t row) {
  int lo = 0, hi = groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ TileRows tile_rows(const Fp4View& v, int q) {
  TileRows t;
  if (!v.offsets) {
    const int group_rows = static_cast<int>(v.group_rows);
    int g = 0, in = q;
    if (v.groups > 1) {
      const int per = (group_rows + kTileRows - 1) / kTileRows;
      g = q / per;
      in = q - g * per;
    }
    t.row = g * group_rows + in * kTileRows;
    t.count = min(kTileRows, group_rows - in * kTileRows);
    t.tile = q;
    return t;
  }
  const int g = find_group(v.offsets, v.groups, kTileRows, q);
  const int first = v.offsets[g];
  const int end = g < v.groups ? v.offsets[g + 1] : static_cast<int>(v.rows);
  t.row = first + (q - (first / kTileRows + g)) * kTileRows;
  t.count = max(min(kTileRows, end - t.row), 0);
  t.tile = g < v.groups ? q : -1;
  return t;
}

// Eight fp32 values, already divided by their scale, to eight E2M1 codes:
// value i in bits 4i .. 4i + 3 (nearest, ties to even, at most 6).
__device__ __forceinline__ uint32_t to_e2m1(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight E2M1 codes to fp32.
__device__ __forceinline__ void from_e2m1(uint32_t codes, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// E4M3 byte of a non-negative value (nearest even, at most 448) ...
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xffu;
}
// ... and back.
__device__ __forceinline__ float from_e4m3(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu)));
}

constexpr uint32_t kNanE4M3 = 0x7f, kNanE8M0 = 0xff;

__device__ __forceinline__ float from_e8m0(uint32_t byte) {
  if (byte == kNanE8M0) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(byte ? byte << 23 : 1u << 22);
}

template <int kFormat>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return kFormat == FP4_NV ? from_e4m3(byte) : from_e8m0(byte);
}

}  // namespace gb300
