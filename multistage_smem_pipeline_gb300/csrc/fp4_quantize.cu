// Quantisation to 4-bit blocks, and back.
//
// Each thread takes 16 neighbouring elements (a block of FP4_NV, half a block
// of FP4_MX).  Both kernels read and write every element once and are bound
// by memory: 2 bytes in and 1/2 + 1/16 (1/32) out per element, or the reverse.
#include "fp4.cuh"

namespace gb300 {
namespace {

constexpr int kSegment = 16;                            // elements a thread takes
constexpr int kTileSegments = kStageCols / kSegment;    // of them across 256 columns
constexpr int kThreads = 256;

// A chunk of scales, 128 rows by 4 blocks, is what a block of threads handles
// in the kernels that go by tiles.
template <int kFormat>
struct Chunk {
  static constexpr int kCols = 4 * block_size(kFormat);         // 64 or 128
  static constexpr int kSegments = kCols / kSegment;            // across it: 4 or 8
  static constexpr int kRowsAtOnce = kThreads / kSegments;      // 64 or 32
  static constexpr int kSteps = kTileRows / kRowsAtOnce;        // 2 or 4
};

// 16 elements of a row as they are stored, from column c on; what lies at
// `cols` or past it is undefined.  kVec: the row is 16-byte aligned.
struct Raw {
  Pack p[2];
};

template <bool kVec>
__device__ __forceinline__ Raw load_raw(const uint16_t* row, int c, int cols) {
  Raw r;
  std::memset(&r, 0, sizeof(r));
  if (kVec && c + kSegment <= cols) {
    r.p[0] = load8<true>(row, c, cols);
    r.p[1] = load8<true>(row, c + 8, cols);
  } else {
    if (c < cols) r.p[0] = load8<false>(row, c, cols);
    if (c + 8 < cols) r.p[1] = load8<false>(row, c + 8, cols);
  }
  return r;
}

// Zeroes the elements at `cols` and past it.
__device__ __forceinline__ void clip(Raw& r, int c, int cols) {
  if (c + kSegment <= cols) return;
#pragma unroll
  for (int i = 0; i < kSegment / 2; ++i) {
    uint32_t& w = r.p[i >> 2].w[i & 3];
    if (c + 2 * i >= cols) w = 0;
    else if (c + 2 * i + 1 >= cols) w &= 0xffffu;
  }
}

// The larger magnitudes of two pairs of elements, each half for itself; a NaN
// in either wins.  The sign is the product of the two's and means nothing.
template <typename T>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t max_pair<__half>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <>
__device__ __forceinline__ uint32_t max_pair<__nv_bfloat16>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two fp32 products, or fused products and sums, in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}

struct Segment {
  uint2 codes;
  uint32_t scale;  // byte
};

// 16 elements to codes and their block's scale.  FP4_MX: called by whole
// warps, the two threads of a block being neighbours.
//
// The quotient must round to E2M1 as the exact one does, ties included, and
// x times the rounded reciprocal does not always: for scales of significand
// 13/8 to 15/8 some exact ties move.  So the reciprocal is held in two parts,
// hi + lo, and the quotient is fma(x, hi, x lo): within 2^-24 of the exact
// one after a single rounding, hence equal to it at a tie (which fp32 holds),
// and never across one, as x and a tie that differ do so by at least 2^-11.
// Checked for every fp16 and bf16 value against every scale.  The powers of
// two of the exponent go into the two parts.
template <typename T, int kFormat>
__device__ __forceinline__ Segment quantize_segment(const Raw& raw, const Fp4View& v) {
  uint32_t both = raw.p[0].w[0];  // largest magnitudes of the even and the odd elements
#pragma unroll
  for (int i = 1; i < kSegment / 2; ++i) both = max_pair<T>(both, raw.p[i >> 2].w[i & 3]);
  both &= 0x7fff7fffu;
  const T* const halves = reinterpret_cast<const T*>(&both);
  // compared as bits, so that a NaN is larger than everything
  uint32_t top = max(__float_as_uint(to_float(halves[0])), __float_as_uint(to_float(halves[1])));
  Segment s;
  float hi, lo = 0.0f;
  bool finite;
  if (kFormat == FP4_NV) {
    // amax / 6 in the same way: 1/6 in two parts
    constexpr float kSixth = 1.0f / 6.0f;
    const float sixth_lo = fmaf(-kSixth, 6.0f, 1.0f) * kSixth;
    const float scaled = __uint_as_float(top) * v.down;
    finite = __float_as_uint(scaled) < 0x7f800000u;
    s.scale = finite ? to_e4m3(fmaf(scaled, kSixth, scaled * sixth_lo)) : kNanE4M3;
    const float step = finite ? from_e4m3(s.scale) : 0.0f;
    // the approximate reciprocal will do: lo makes up for what it is off by
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(hi) : "f"(step));
    if (!(step > 0.0f)) hi = 0.0f;
    lo = fmaf(-hi, step, 1.0f) * hi * v.down;
    hi *= v.down;
  } else {
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const int field = static_cast<int>(top >> 23);
    finite = field != 0xff;
    s.scale = finite ? static_cast<uint32_t>(max(field - 2, 0)) : kNanE8M0;
    hi = finite ? __uint_as_float((254u - s.scale) << 23) : 0.0f;
  }
  float q[kSegment];
#pragma unroll
  for (int i = 0; i < kSegment; i += 2) {
    const T* const e = reinterpret_cast<const T*>(&raw.p[i >> 3].w[(i >> 1) & 3]);
    const float2 x = make_float2(to_float(e[0]), to_float(e[1]));
    float2 y;
    if (kFormat == FP4_NV) y = fma2(x, make_float2(hi, hi), mul2(x, make_float2(lo, lo)));
    else y = mul2(x, make_float2(hi, hi));
    q[i] = y.x;
    q[i + 1] = y.y;
  }
  s.codes = finite ? make_uint2(to_e2m1(q), to_e2m1(q + 8)) : make_uint2(0, 0);
  return s;
}

// Codes and their block's scale to 16 elements.
template <typename T, int kFormat>
__device__ __forceinline__ void dequantize_segment(Pack (&p)[2], uint2 codes, uint32_t scale,
                                                   const Fp4View& v) {
  float f[kSegment];
  from_e2m1(codes.x, f);
  from_e2m1(codes.y, f + 8);
  const float step = scale_value<kFormat>(scale) * (kFormat == FP4_NV ? v.up : 1.0f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float half[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) half[e] = f[8 * h + e] * step;
    p[h] = pack<T>(half);
  }
}

// A block per chunk, going down the tiles.  All of a thread's rows of a tile
// are asked for before the first is used; the chunk is put together in shared
// memory and written in one piece.  Six blocks an SM for FP4_NV and four for
// FP4_MX (twice the rows in flight a thread) are what their registers are held
// to: 8192 x 8192 nvfp4 takes 28 us against 33 without (6.1 TB/s); asking for
// the next tile as well was slower for the registers it took (38).
template <typename T, int kFormat, bool kVec>
__global__ void __launch_bounds__(kThreads, kFormat == FP4_NV ? 6 : 4)
    quantize_kernel(const Fp4View v, const uint16_t* __restrict__ x, int64_t ldx, int tiles) {
  using C = Chunk<kFormat>;
  __shared__ __align__(16) uint8_t scales[kChunkBytes];
  grid_launch_dependents();
  const int cols = static_cast<int>(v.cols);
  const int seg = threadIdx.x % C::kSegments;
  const int c = static_cast<int>(blockIdx.x) * C::kCols + seg * kSegment;
  const int r0 = threadIdx.x / C::kSegments;
  const bool padded = c / 2 < static_cast<int>(v.pitch);
  grid_dependency_wait();
  for (int tile = blockIdx.y; tile < tiles; tile += gridDim.y) {
    const TileRows t = tile_rows(v, tile);
    Raw raw[C::kSteps];
    const uint16_t* from = x + (t.row + r0) * ldx;
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) {
      raw[i] = load_raw<kVec>(from, c, r0 + i * C::kRowsAtOnce < t.count ? cols : 0);
      from += C::kRowsAtOnce * ldx;
    }
    if (threadIdx.x < kChunkBytes / 16)
      reinterpret_cast<uint4*>(scales)[threadIdx.x] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    uint8_t* to = v.codes + (t.row + r0) * v.pitch + c / 2;
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) {
      const int r = r0 + i * C::kRowsAtOnce;
      if (i * C::kRowsAtOnce >= t.count) break;
      clip(raw[i], c, cols);
      const Segment s = quantize_segment<T, kFormat>(raw[i], v);
      if (r < t.count) {
        if (padded) *reinterpret_cast<uint2*>(to) = s.codes;
        if (c < cols) scales[scale_at(r, kFormat == FP4_NV ? seg : seg >> 1)] = s.scale;
      }
      to += C::kRowsAtOnce * v.pitch;
    }
    __syncthreads();
    if (threadIdx.x < kChunkBytes / 16)
      reinterpret_cast<uint4*>(v.scales + t.tile * v.tile_bytes +
                               static_cast<int64_t>(blockIdx.x) * kChunkBytes)[threadIdx.x] =
          reinterpret_cast<const uint4*>(scales)[threadIdx.x];
  }
}

// A block per token and up to 4096 columns: quantised once, written to the row
// of each of its kept slots, whose places the first threads look up: the expert
// of a row is the group it lies in, found among the offsets in shared memory
// (one latency for all of them).  The caller's list of experts would be a shorter
// way to it (4096 tokens of 2880 into 2 slots each of 8 experts 7.5 us, so 8.4; 4096
// of 4096 into 8 of 64 22.5 and 22.3), but may hold the next step's by now.
// Neighbouring threads join the four scale bytes of a chunk.  4096 tokens of
// 4096 columns into 8 slots each take 22.3 us (4.9 TB/s); what it waits on are
// the scales, 4 bytes of a row in each 512-byte chunk, as writing codes 16 bytes
// a thread instead of 8 changed nothing.
template <typename T, int kFormat, bool kVec>
__global__ void __launch_bounds__(kThreads)
    quantize_routed_kernel(const Fp4View v, const uint16_t* __restrict__ x, int64_t ldx,
                           const int32_t* __restrict__ rows, int top_k) {
  constexpr int kPerBlock = kFormat == FP4_NV ? 1 : 2;
  __shared__ int64_t s_codes[MOE_MAX_TOP_K], s_scales[MOE_MAX_TOP_K];  // -1: dropped
  __shared__ int32_t s_first[MOE_MAX_EXPERTS + 1];
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t token = blockIdx.x;
  const int cols = static_cast<int>(v.cols);
  const int seg = static_cast<int>(blockIdx.y) * kThreads + threadIdx.x;
  const int c = seg * kSegment;
  Raw raw = load_raw<kVec>(x + token * ldx, c, cols);
  for (int g = threadIdx.x; g <= v.groups; g += kThreads) s_first[g] = v.offsets[g];
  const int32_t row = threadIdx.x < top_k ? rows[token * top_k + threadIdx.x] : -1;
  __syncthreads();
  if (threadIdx.x < top_k) {
    int64_t codes = -1;
    if (row >= 0 && row < s_first[v.groups]) {
      const int e = group_of_row(s_first, v.groups, row);
      const int32_t first = s_first[e];
      codes = row * v.pitch;
      s_scales[threadIdx.x] = (first / kTileRows + e + (row - first) / kTileRows) * v.tile_bytes +
                              scale_at((row - first) % kTileRows, 0);
    }
    s_codes[threadIdx.x] = codes;
  }
  clip(raw, c, cols);
  const Segment s = quantize_segment<T, kFormat>(raw, v);
  // bytes of the chunk's four blocks, in every thread
  uint32_t word = (c < cols ? s.scale : 0u) << (8 * (seg / kPerBlock & 3));
  if (kFormat == FP4_MX && (seg & 1)) word = 0;
#pragma unroll
  for (int d = 1; d < 4 * kPerBlock; d <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, d);
  __syncthreads();
  if (c >= static_cast<int>(col_stages(v.cols)) * kStageCols) return;
  const bool padded = c / 2 < static_cast<int>(v.pitch);
  const bool leads = seg % (4 * kPerBlock) == 0;
  uint8_t* const codes = v.codes + c / 2;
  uint8_t* const scales = v.scales + static_cast<int64_t>(seg / (4 * kPerBlock)) * kChunkBytes;
#pragma unroll 4
  for (int j = 0; j < top_k; ++j) {
    const int64_t at = s_codes[j];
    if (at < 0) continue;
    if (padded) *reinterpret_cast<uint2*>(codes + at) = s.codes;
    if (leads) *reinterpret_cast<uint32_t*>(scales + s_scales[j]) = word;
  }
}

// A block per chunk and tile, or 128 rows of no group, going down them.  8192 x
// 8192 nvfp4 to bf16 in 28 us (6.1 TB/s).
template <typename T, int kFormat>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(uint16_t* __restrict__ y, const Fp4View v, int tiles) {
  using C = Chunk<kFormat>;
  __shared__ __align__(16) uint8_t scales[kChunkBytes];
  grid_launch_dependents();
  grid_dependency_wait();
  const int cols = static_cast<int>(v.cols);
  const int seg = threadIdx.x % C::kSegments;
  const int c = static_cast<int>(blockIdx.x) * C::kCols + seg * kSegment;
  const int r0 = threadIdx.x / C::kSegments;
  for (int tile = blockIdx.y; tile < tiles; tile += gridDim.y) {
    const TileRows t = tile_rows(v, tile);
    if (t.count == 0) continue;
    __syncthreads();  // the last tile's scales have been read
    uint2 codes[C::kSteps];
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) {
      const int r = r0 + i * C::kRowsAtOnce;
      codes[i] = make_uint2(0, 0);
      if (t.tile >= 0 && r < t.count && c < cols)
        codes[i] = *reinterpret_cast<const uint2*>(v.codes + static_cast<int64_t>(t.row + r) * v.pitch + c / 2);
    }
    if (t.tile >= 0 && threadIdx.x < kChunkBytes / 16)
      reinterpret_cast<uint4*>(scales)[threadIdx.x] = reinterpret_cast<const uint4*>(
          v.scales + t.tile * v.tile_bytes + static_cast<int64_t>(blockIdx.x) * kChunkBytes)[threadIdx.x];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) {
      if (i * C::kRowsAtOnce >= t.count) break;
      const int r = r0 + i * C::kRowsAtOnce;
      Pack p[2] = {};
      if (t.tile >= 0)
        dequantize_segment<T, kFormat>(p, codes[i],
                                       scales[scale_at(r, kFormat == FP4_NV ? seg : seg >> 1)], v);
      // Neighbours swap halves, so that a warp's store covers 32-byte sectors
      // whole: first both halves of the even segment, then of the odd one.
      const bool odd = seg & 1;
      Pack other;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        other.w[w] = __shfl_xor_sync(0xffffffffu, odd ? p[0].w[w] : p[1].w[w], 1);
      if (r >= t.count) continue;
      uint16_t* const row = y + (t.row + r) * v.cols;
      const int even = c - (odd ? kSegment : 0);  // cols is a multiple of 8: pieces are whole
      const int first = even + (odd ? 8 : 0), second = first + kSegment;
      if (first < cols) store8<true>(row, first, cols, odd ? other : p[0]);
      if (second < cols) store8<true>(row, second, cols, odd ? p[1] : other);
    }
  }
}

// Rows that start anywhere.  A block takes 16 rows of 256 columns at a time, so
// that there are blocks enough for the smaller matrices and few ends of rows, and
// puts them together in shared memory; from there they leave in windows of 16
// bytes that are aligned in the output's row, and what lies before the first and
// after the last one by one.  The next rows are asked for before that.  2411 x
// 1169 mxfp4 to fp16 in 3.3 us, where blocks of a whole tile that store single
// elements take 8.6 (aligned, 1168: 3.5); 8191 x 8191 nvfp4 in 41 (4.2 TB/s; by
// whole tiles 47, aligned 28), bound by instruction issue: shifts and rows' ends.
template <typename T, int kFormat>
__global__ void __launch_bounds__(kThreads)
    dequantize_unaligned_kernel(uint16_t* __restrict__ y, const Fp4View v, int64_t steps) {
  constexpr int kRows = kThreads / kTileSegments;  // 16
  constexpr int kSteps = kTileRows / kRows;        // to a tile
  constexpr int kWindows = kStageCols / 8;         // of a row, at most
  __shared__ __align__(16) uint16_t staged[kRows * kStageCols + 8];  // 8: read past the last
  grid_launch_dependents();
  grid_dependency_wait();
  const int cols = static_cast<int>(v.cols);
  const int seg = threadIdx.x % kTileSegments;
  const int c0 = static_cast<int>(blockIdx.x) * kStageCols;
  const int c = c0 + seg * kSegment;
  const int r0 = threadIdx.x / kTileSegments;
  const int here = min(kStageCols, cols - c0);
  struct Rows {
    int first, count;  // of the matrix, and how many (none: 0 or less)
    bool live;         // this thread's segment has codes
    uint2 codes;
    uint32_t scale;
  };
  const auto load = [&](int64_t step) {
    Rows n;
    n.count = 0;
    n.live = false;
    if (step >= steps) return n;
    const TileRows t = tile_rows(v, static_cast<int>(step / kSteps));
    const int in = static_cast<int>(step % kSteps) * kRows;
    n.first = t.row + in;
    n.count = min(kRows, t.count - in);
    n.live = t.tile >= 0 && r0 < n.count && c < cols;
    if (n.live) {
      n.codes = *reinterpret_cast<const uint2*>(v.codes + (n.first + r0) * v.pitch + c / 2);
      const int64_t at = t.tile * v.tile_bytes +
                         static_cast<int64_t>(blockIdx.x) * chunks_per_stage(kFormat) * kChunkBytes;
      n.scale = v.scales[at + scale_at(in + r0, kFormat == FP4_NV ? seg : seg >> 1)];
    }
    return n;
  };
  Rows next = load(blockIdx.y);
  for (int64_t step = blockIdx.y; step < steps; step += gridDim.y) {
    const Rows now = next;
    next = load(step + gridDim.y);
    if (now.count <= 0) continue;
    Pack p[2] = {};
    if (now.live) dequantize_segment<T, kFormat>(p, now.codes, now.scale, v);
    __syncthreads();  // the last rows have left
    *reinterpret_cast<Pack*>(staged + r0 * kStageCols + seg * kSegment) = p[0];
    *reinterpret_cast<Pack*>(staged + r0 * kStageCols + seg * kSegment + 8) = p[1];
    __syncthreads();
    uint16_t* const to = y + now.first * v.cols + c0;
    for (int r = threadIdx.x / kWindows; r < now.count; r += kThreads / kWindows) {
      uint16_t* const row = to + r * v.cols;
      const int head = -row_lead(row) & 7, at = threadIdx.x % kWindows * 8;
      if (at + head + 8 > here) continue;
      const uint4* const from = reinterpret_cast<const uint4*>(staged + r * kStageCols + at);
      *reinterpret_cast<Pack*>(row + at + head) = shift8(from[0], from[1], 2 * head);
    }
    if (threadIdx.x < now.count * 16) {
      const int r = threadIdx.x / 16, k = threadIdx.x % 8;
      const bool ahead = threadIdx.x % 16 < 8;
      uint16_t* const row = to + r * v.cols;
      const int head = min(-row_lead(row) & 7, here);
      const int tail = head + (here - head) / 8 * 8;  // past the last whole window
      const int e = ahead ? k : tail + k;
      if (e < (ahead ? head : here)) row[e] = staged[r * kStageCols + e];
    }
  }
}

// Blocks for every chunk of every tile, up to 24 an SM (and no more rows of them
// than a grid may have): each goes down the tiles in that stride.
dim3 tile_grid(int64_t chunks, int64_t tiles, int sms) {
  const int64_t rows = std::min<int64_t>(std::max<int64_t>(24 * sms / chunks, 1), 65535);
  return dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(std::min(tiles, rows)));
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
  if (any_overlap({{x, xbytes, false},
                   {out->codes, code_bytes(out), true},
                   {out->scales, scale_bytes(out), true}},
                  routing))
    return GEMM_ERR_INVALID_VALUE;
  int sms = 0;
  if ((rc = require_device(&sms)) != GEMM_OK) return rc;
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
      return launch_pdl(quantize_routed_kernel<T, fmt(), wide()>, grid, dim3(kThreads), 0, s, 1u, v, xp,
                        ldx, routing->rows, routing->top_k);
    }
    const int64_t tiles = tile_count(out->rows, out->groups, false);
    const int64_t chunks = col_stages(out->cols) * chunks_per_stage(fmt());
    return launch_pdl(quantize_kernel<T, fmt(), wide()>, tile_grid(chunks, tiles, sms), dim3(kThreads), 0,
                      s, 1u, v, xp, ldx, static_cast<int>(tiles));
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
  if (any_overlap({{y, ybytes, true},
                   {in->codes, code_bytes(in), false},
                   {in->scales, scale_bytes(in), false},
                   {in->offsets, offset_bytes(in), false}}))
    return GEMM_ERR_INVALID_VALUE;
  int sms = 0;
  if ((rc = require_device(&sms)) != GEMM_OK) return rc;
  const Fp4View v = view_of(in);
  const bool vec = aligned_to(y, 16) && in->cols % 8 == 0;
  const bool by_offsets = in->offsets != nullptr;
  return dispatch_forms(type, in->format, vec, [&](auto t, auto fmt, auto wide) {
    using T = decltype(t);
    const int64_t tiles = tile_count(in->rows, in->groups, by_offsets) + (by_offsets ? 1 : 0);
    uint16_t* const to = static_cast<uint16_t*>(y);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (wide()) {
      // only the columns that y has: padding is left out
      const int64_t chunks = (in->cols + Chunk<fmt()>::kCols - 1) / Chunk<fmt()>::kCols;
      return launch_pdl(dequantize_kernel<T, fmt()>, tile_grid(chunks, tiles, sms), dim3(kThreads), 0,
                        s, 1u, to, v, static_cast<int>(tiles));
    }
    const int64_t steps = tiles * (kTileRows * kTileSegments / kThreads);
    return launch_pdl(dequantize_unaligned_kernel<T, fmt()>,
                      tile_grid(col_stages(in->cols), steps, sms), dim3(kThreads), 0, s, 1u, to, v,
                      steps);
  });
}
