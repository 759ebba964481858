// Host side of fp4_gemm_tn: checks, the choice of tile, tensor maps, launch.
#include <cuda.h>

#include <cmath>
#include <mutex>

#include "fp4_gemm_pair_kernel.cuh"

namespace gb300 {
namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull;

// A matrix's codes as rows of bytes; a box is 128 bytes wide.
int encode_codes(EncodeTiledFn encode, CUtensorMap* map, const fp4_matrix_t* m, uint32_t box_rows) {
  const uint64_t pitch = static_cast<uint64_t>(code_pitch(m->cols));
  const cuuint64_t dims[2] = {pitch, static_cast<cuuint64_t>(m->rows)};
  const cuuint64_t strides[1] = {pitch};
  const cuuint32_t box[2] = {kGemmBytesK, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m->codes, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

// A matrix's scales as rows of one chunk, 128 words; a box is a stage's chunks.
int encode_scales(EncodeTiledFn encode, CUtensorMap* map, const fp4_matrix_t* m, int64_t chunks) {
  const cuuint64_t dims[2] = {kChunkBytes / 4, static_cast<cuuint64_t>(chunks)};
  const cuuint64_t strides[1] = {kChunkBytes};
  const cuuint32_t box[2] = {kChunkBytes / 4,
                             static_cast<cuuint32_t>(chunks_per_stage(m->format))};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, m->scales, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

template <typename T, int kFormat, bool kSplit>
int launch_single(const CUtensorMap& w, const CUtensorMap& x, Fp4GemmParams p, int tiles,
                  int device, cudaStream_t s) {
  const uint32_t fixed = gemm_fixed_bytes(p.offsets ? p.groups : 0) + (kSplit ? kSplitBytes : 0u);
  using S = Fp4GemmShape<kFormat>;
  p.stages = S::stages_that_fit(fixed);
  const auto kernel = fp4_gemm_tc<T, kFormat, kSplit>;
  static std::atomic<uint64_t> granted{0};  // per instantiation
  if (!grant_smem(kernel, kGemmSmemLimit, device, granted)) return GEMM_ERR_CUDA;
  return launch_pdl(kernel, dim3(tiles * p.split), dim3(kGemmThreads),
                    fixed + p.stages * S::kStageBytes, s, static_cast<unsigned>(p.split), w, x, p);
}

int machine_of(int sms, int device, Machine* machine) {
  static PerDevice<Machine> known;
  return machine_by(fp4_gemm_tc<__half, FP4_NV, true>, kGemmThreads, kGemmSmemLimit, sms, device,
                    known, machine);
}

// CTAs that share each of `tiles` tiles' k.  Measured on GB300: a 256-column
// block of k takes a lone CTA about 0.28 us (the latency of its loads), and
// meeting the others 0.6 us and, for the partial sums, up to 3 us for 128 rows.
// Weights from memory, by one and by two, four or eight: 1 x 4096 x 14336 16.9 us and
// 12.7, 9.9, -; 128 x 128 x 32768 35.4 and 23.7, 15.4, 9.8; 128 x 512 x 1024, from
// cache, 4.7 and 8.3.  All of the clusters have to fit at once (16 tiles by eight:
// 12.0 us where four take 7.5).
int choose_split(int64_t tiles, int64_t rows, int num_kb, const Machine& machine) {
  int best = 1;
  double least = 0.28 * num_kb;
  for (int i = 0; i < 3 && 4 << i <= num_kb && tiles <= machine.clusters[i]; ++i) {
    const int split = 2 << i;
    const double t = 0.28 * num_kb / split + 0.6 + 3.0 * std::min<int64_t>(rows, 128) / 128;
    if (t < least) {
      least = t;
      best = split;
    }
  }
  return best;
}

struct Plan {
  bool pair;
  int tile;           // outputs and rows of one
  int m_tiles;        // of a group
  int box_rows;
  int split;
  int units;          // CTAs, pairs or clusters
  int64_t x_chunks, w_chunks;
};

// The form of a product of `rows` rows in `groups` groups with `n` outputs each:
// 128 x 128 tiles on single CTAs, those tiles' k shared by clusters, or 256 x 256
// on pairs.  Where single CTAs have a tile each at most, they are it, split where
// there are few: pairs would leave more SMs idle (256 x 8192 x 14336: 22.4 us where
// single CTAs take 19.5; 1 x 4096 x 14336: 17.8, 16.9, and 9.9 split).  Past
// that, whichever's waves of tiles take fewer cycles: a tile takes a single CTA about
// 1200 + 580 per 256 columns of k, and a pair, four times the work, 4500 + 500,
// with one accumulator, so that a tile's stores are not all hidden (8192^3: 261 us
// by single CTAs, 164 by pairs; 8192 x 4096 x 256: 16 and 24).  With groups by
// offsets the number of row tiles is not known here: a group is taken to end half
// way through its last.  150 dense shapes (1 to 512 rows, 128 to 8192 outputs, k
// 2048 to 32768, weights from memory) take 0.8 % over the best form of each in the
// mean, at worst 30 (16 x 8192 x 2048: 7.3 us by two, 5.6 by one).
int make_plan(int64_t rows, int64_t n, int64_t cols, int format, int64_t groups, bool by_offsets,
              const Machine& machine, Plan* o) {
  const int num_kb = static_cast<int>(col_stages(cols));
  const int64_t group_rows = by_offsets ? 0 : rows / groups;
  const int64_t tile_chunks = static_cast<int64_t>(num_kb) * chunks_per_stage(format);
  const int64_t live = std::min(groups, rows);
  const auto m_tiles = [&](int64_t tile) { return (n + tile - 1) / tile; };
  const auto expected = [&](int64_t tile) {  // tiles
    return m_tiles(tile) * (by_offsets ? std::max(live, (2 * rows + live * tile) / (2 * tile))
                                       : groups * ((group_rows + tile - 1) / tile));
  };
  const auto most = [&](int64_t tile) {
    return m_tiles(tile) *
           (by_offsets ? rows / tile + live : groups * ((group_rows + tile - 1) / tile));
  };
  // rows of a tile, in the mean: of the groups that there can be
  const int64_t tile_rows =
      by_offsets ? (rows + groups - 1) / groups : std::min<int64_t>(group_rows, 128);
  // counted in 32 bits by the kernel over pairs
  o->x_chunks = tile_count(rows, groups, by_offsets) * tile_chunks;
  o->w_chunks = groups * ((n + kTileRows - 1) / kTileRows) * tile_chunks;
  const auto waves = [&](int64_t tile, int64_t slots) { return (expected(tile) + slots - 1) / slots; };
  o->pair = waves(128, machine.sms) > 1 &&
            waves(256, machine.sms / 2) * (4500 + 500 * num_kb) <
                waves(128, machine.sms) * (1200 + 580 * num_kb) &&
            o->x_chunks <= INT_MAX && o->w_chunks <= INT_MAX;
  o->split = o->pair ? 1 : choose_split(most(128), tile_rows, num_kb, machine);
  o->tile = o->pair ? 256 : 128;
  // counted in 32 bits, with room for a grid's stride past the last
  if (most(o->tile) > INT_MAX / 4) return GEMM_ERR_INVALID_VALUE;
  o->m_tiles = static_cast<int>(m_tiles(o->tile));
  // Boxes of 32 rows where a group may end anywhere in a tile, so that a tile
  // loads little more than it has (8 tokens over 64 experts: 21 us against 27
  // with boxes of 128).
  o->box_rows = by_offsets || group_rows <= 64 ? 32 : 128;
  // One CTA per SM, fewer where there cannot be that many tiles.
  o->units = static_cast<int>(
      std::min<int64_t>(o->pair ? machine.sms / 2 : machine.sms, most(o->tile)));
  return GEMM_OK;
}

struct PairMaps {
  CUtensorMap w, x, sw, sx;
};

template <typename T, int kFormat>
int launch_pair(const PairMaps& m, Fp4GemmParams p, int pairs, int device, cudaStream_t s) {
  const uint32_t fixed = gemm_fixed_bytes(p.offsets ? p.groups : 0);
  using S = Fp4PairShape<kFormat>;
  p.stages = S::stages_that_fit(fixed);
  static std::atomic<uint64_t> granted{0};  // per instantiation
  if (!grant_smem(fp4_gemm_pair<T, kFormat>, kGemmSmemLimit, device, granted)) return GEMM_ERR_CUDA;
  return launch_pdl(fp4_gemm_pair<T, kFormat>, dim3(2 * pairs), dim3(kGemmThreads),
                    fixed + S::ring_bytes(p.stages), s, 2u, m.w, m.x, m.sw, m.sx, p);
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" int fp4_gemm_tn(void* D, int type, const fp4_matrix_t* a, const fp4_matrix_t* b,
                           float alpha, void* stream) {
  return fp4_gemm_tn_ex(D, type, a, b, alpha, 0, 0, stream);
}

extern "C" int fp4_gemm_tn_ex(void* D, int type, const fp4_matrix_t* a, const fp4_matrix_t* b,
                              float alpha, uint64_t timeout_ns, int inject, void* stream) {
  bool any_a = false, any_b = false;
  int rc = check_matrix(a, &any_a);
  if (rc != GEMM_OK) return rc;
  if ((rc = check_matrix(b, &any_b)) != GEMM_OK) return rc;
  if (!valid_type(type) || !std::isfinite(alpha) || inject < 0 || inject > 1 || a->format != b->format || a->cols != b->cols ||
      a->groups != b->groups || b->offsets)
    return GEMM_ERR_INVALID_VALUE;
  const double scale = std::ldexp(static_cast<double>(alpha), a->exponent + b->exponent);
  if (!std::isfinite(static_cast<float>(scale))) return GEMM_ERR_INVALID_VALUE;
  const int64_t n_out = b->group_rows;
  if (a->rows == 0 || n_out == 0) return GEMM_OK;
  if (!D) return GEMM_ERR_INVALID_VALUE;
  if (!aligned_to(D, 2)) return GEMM_ERR_MISALIGNED;
  const uint64_t dbytes = static_cast<uint64_t>(a->rows) * n_out * 2;
  for (const fp4_matrix_t* m : {a, b})
    if (any_overlap({{D, dbytes, true},
                     {m->codes, code_bytes(m), false},
                     {m->scales, scale_bytes(m), false},
                     {m->offsets, offset_bytes(m), false}}))
      return GEMM_ERR_INVALID_VALUE;
  int sms = 0, device = 0;
  if ((rc = require_device(&sms, &device)) != GEMM_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->cols == 0) return write_empty_sum(D, nullptr, 0.0f, a->rows * n_out, sms, s);
  EncodeTiledFn encode = nullptr;
  if ((rc = get_encoder(&encode)) != GEMM_OK) return rc;

  Fp4GemmParams p;
  std::memset(&p, 0, sizeof(p));
  const Fp4View va = view_of(a), vb = view_of(b);
  p.w_scales = vb.scales;
  p.x_scales = va.scales;
  p.w_tile_bytes = vb.tile_bytes;
  p.x_tile_bytes = va.tile_bytes;
  p.d = static_cast<uint16_t*>(D);
  p.offsets = a->offsets;
  p.rows = a->rows;
  p.group_rows = a->group_rows;
  p.n_out = n_out;
  p.groups = a->groups;
  p.num_kb = static_cast<int32_t>(col_stages(a->cols));
  p.w_group_tiles = static_cast<int32_t>((n_out + kTileRows - 1) / kTileRows);
  p.tile_chunks = p.num_kb * chunks_per_stage(a->format);
  // One rounding, whatever the exponents' order.  Below fp32's normal numbers the
  // factor would lose bits or be zero where the results need not be (sums reach
  // 2^46): then it is applied in two steps, 2^120 times the factor and 2^-120.
  const bool tiny = std::fabs(scale) < std::ldexp(1.0, -126);
  p.pre = tiny ? static_cast<float>(std::ldexp(scale, 120)) : 1.0f;
  p.alpha = tiny ? power_of_two(-120) : static_cast<float>(scale);
  p.timeout_ns = timeout_ns ? timeout_ns : kTimeoutNs;
  p.inject = inject;
  p.error_word = error_index(s);

  Machine machine;
  if ((rc = machine_of(sms, device, &machine)) != GEMM_OK) return rc;
  Plan plan;
  rc = make_plan(a->rows, n_out, a->cols, a->format, a->groups, a->offsets != nullptr, machine,
                 &plan);
  if (rc != GEMM_OK) return rc;
  p.m_tiles = plan.m_tiles;
  p.box_rows = plan.box_rows;
  p.split = plan.split;
  PairMaps m;
  if ((rc = encode_codes(encode, &m.w, b, kGemmM)) != GEMM_OK ||
      (rc = encode_codes(encode, &m.x, a, p.box_rows)) != GEMM_OK)
    return rc;
  if (plan.pair && ((rc = encode_scales(encode, &m.sw, b, plan.w_chunks)) != GEMM_OK ||
                    (rc = encode_scales(encode, &m.sx, a, plan.x_chunks)) != GEMM_OK))
    return rc;
  const auto go = [&](auto t, auto fmt) {
    using T = decltype(t);
    if (plan.pair) return launch_pair<T, fmt()>(m, p, plan.units, device, s);
    return p.split > 1 ? launch_single<T, fmt(), true>(m.w, m.x, p, plan.units, device, s)
                       : launch_single<T, fmt(), false>(m.w, m.x, p, plan.units, device, s);
  };
  const auto by_format = [&](auto t) {
    return a->format == FP4_NV ? go(t, std::integral_constant<int, FP4_NV>{})
                               : go(t, std::integral_constant<int, FP4_MX>{});
  };
  return type == MOE_F16 ? by_format(__half{}) : by_format(__nv_bfloat16{});
}

extern "C" int fp4_query_config(int64_t rows, int64_t n, int64_t cols, int format, int groups,
                                int by_offsets, fp4_config_t* out) {
  if (!out || rows < 1 || n < 1 || cols < 1 || !fits(rows, cols) || check_format(format) != GEMM_OK ||
      groups < 1 || (by_offsets != 0 && by_offsets != 1) ||
      (by_offsets ? groups > MOE_MAX_EXPERTS : rows % groups != 0) || n > INT_MAX / groups)
    return GEMM_ERR_INVALID_VALUE;
  Machine machine{152, {76, 36, 15}};
  int sms = 0, device = 0, rc = GEMM_OK;
  if (require_device(&sms, &device) != GEMM_OK) cudaGetLastError();
  else if ((rc = machine_of(sms, device, &machine)) != GEMM_OK) return rc;
  Plan plan;
  rc = make_plan(rows, n, cols, format, groups, by_offsets != 0, machine, &plan);
  if (rc != GEMM_OK) return rc;
  *out = fp4_config_t{plan.pair ? 1 : 0, plan.split, plan.tile, plan.box_rows,
                      plan.units * (plan.pair ? 2 : plan.split)};
  return GEMM_OK;
}

extern "C" int fp4_get_device_error(void* stream, uint32_t* raw) {
  const int rc = require_device(nullptr);
  if (rc != GEMM_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  const uint32_t zero = 0;
  const size_t off = static_cast<size_t>(error_index(s)) * sizeof(uint32_t);
  if (cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&word, g_fp4_error, sizeof(word), off, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_fp4_error, &zero, sizeof(zero), off, cudaMemcpyHostToDevice, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (raw) *raw = word;
  return static_cast<int>(word & 0xffu);
}
