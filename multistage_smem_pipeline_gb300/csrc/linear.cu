// Host side of linear layers: checks, workspaces, the form of a product, tensor
// maps, launches.
#include <cmath>

#include "linear_few_kernel.cuh"
#include "linear_kernel.cuh"
#include "linear_pair_kernel.cuh"
#include "linear_rows.cuh"

namespace gb300 {
namespace {

// The limit of a wait that the caller leaves open.  One CTA takes 0.2 us for 64 of a sum, and some
// waits are for a whole sum: that of 2^30 rows of one expert takes 3.3 s.
constexpr uint64_t kTimeoutNs = 2000000000ull, kTimeoutNsPerBlock = 1000;

// ------------------------------------------------------------------ checks
bool in_range(int64_t v, int64_t most) { return v >= 0 && v <= most; }

int groups_of(const linear_t* l) { return l->routing ? l->routing->experts : 1; }

// The stride of a single row does not matter: one that the tensor maps take.
Rows matrix_of(const void* ptr, int64_t rows, int64_t cols, int64_t ld) {
  return Rows{ptr, rows, cols, rows > 1 ? ld : copy_ld(cols)};
}
Rows x_rows(const linear_t* l) { return matrix_of(l->x, l->rows, l->in, l->ldx); }
Rows w_rows(const linear_t* l) { return matrix_of(l->w, groups_of(l) * l->out, l->in, l->ldw); }
Rows by_out(const linear_t* l, const void* ptr, int64_t ld) {
  return matrix_of(ptr, l->rows, l->out, ld);
}

uint64_t bytes_of(const Rows& r) {
  return r.rows && r.cols ? (static_cast<uint64_t>(r.rows - 1) * r.ld + r.cols) * 2 : 0;
}
Range reads(const Rows& r) { return Range{r.ptr, bytes_of(r), false}; }

// A matrix that a call needs; none of its elements: any pointer.
int check_rows(const Rows& r) {
  if (r.ld < r.cols || r.ld > (int64_t{1} << 38)) return GEMM_ERR_INVALID_VALUE;
  if (r.rows == 0 || r.cols == 0) return GEMM_OK;
  if (!r.ptr) return GEMM_ERR_INVALID_VALUE;
  return aligned_to(r.ptr, 2) ? GEMM_OK : GEMM_ERR_MISALIGNED;
}

int check_layer(const linear_t* l) {
  if (!l || !in_range(l->rows, LINEAR_MAX_ROWS) || !in_range(l->in, LINEAR_MAX_COLS) ||
      !in_range(l->out, LINEAR_MAX_COLS) || !valid_type(l->type) || l->activation < LINEAR_NONE ||
      l->activation > LINEAR_SILU)
    return GEMM_ERR_INVALID_VALUE;
  if (l->routing) {
    const int rc = check_routing(l->routing);
    if (rc != GEMM_OK) return rc;
    if (l->rows != l->routing->tokens * l->routing->top_k) return GEMM_ERR_INVALID_VALUE;
  }
  return groups_of(l) * l->out <= INT_MAX ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

// `product`: LINEAR_*, or -1 for any.
bool valid_form(int product, int pair, int tile, int split) {
  if (pair) return pair == 1 && tile == 256 && split == 1;
  if (split != 1 && split != 2 && split != 4 && split != 8) return false;
  if (tile == 1 || tile == 2 || tile == 4 || tile == 8) return product <= LINEAR_FORWARD;
  return tile == 64 || tile == 128 || tile == 256 || (tile == 32 && product != LINEAR_GRAD_W);
}

int check_options(const linear_options_t* o) {
  if (!o) return GEMM_OK;
  if (o->inject < 0 || o->inject > 1) return GEMM_ERR_INVALID_VALUE;
  if (o->tile == 0 && o->cta_pair == 0 && o->split_k == 0) return GEMM_OK;
  return valid_form(-1, o->cta_pair, o->tile, o->split_k) ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

// The offsets of a layer's groups; null for one group (and for rows of nobody).
const int32_t* offsets_of(const linear_t* l) {
  return l->routing && l->rows > 0 ? l->routing->offsets : nullptr;
}

// ------------------------------------------------------------------ forms
int machine_of(int sms, int device, Machine* machine) {
  static PerDevice<Machine> known;
  return machine_by(linear_tc<__half, LINEAR_FORWARD, true, 2>, kLinThreads, kLinSmemLimit, sms,
                    device, known, machine);
}

struct Plan {
  bool pair;
  int tile, split;       // tile up to 8: linear_few
  int m_tiles, n_tiles;  // n_tiles: grad_w's, of a group
  int box_rows;
  int units;             // CTAs, pairs or clusters
};

// A product as the tensor cores see it: m by n, n over all groups but for grad_w, whose
// sums (k) are; `ragged`: groups by offsets.
struct Product {
  int kind;
  int64_t m, n, k;
  int64_t groups;
  bool ragged;
};

Product product_of(int kind, int64_t rows, int64_t in, int64_t out, int64_t groups, bool ragged) {
  switch (kind) {
    case LINEAR_FORWARD: return Product{kind, out, rows, in, groups, ragged};
    case LINEAR_GRAD_X: return Product{kind, in, rows, out, groups, ragged};
    default: return Product{kind, in, out, rows, groups, ragged};
  }
}

Product forward_of(const linear_t* l) {
  return product_of(LINEAR_FORWARD, l->rows, l->in, l->out, groups_of(l), offsets_of(l) != nullptr);
}

// Tiles of N of all groups: as many as are expected, or as there can be.
int64_t n_tiles(const Product& p, int64_t tile, bool most) {
  if (p.kind == LINEAR_GRAD_W) return p.groups * ((p.n + tile - 1) / tile);
  if (!p.ragged) return (p.n + tile - 1) / tile;
  const int64_t live = std::min(p.groups, p.n);
  if (most) return p.n / tile + live;
  // of groups whose sizes are spread as the intervals of a random process are
  return std::llround(live / (1.0 - std::exp(-static_cast<double>(tile) * live / p.n)));
}

// The rows that linear_few takes at a time, where the product is its: by sizes alone, so
// that the workspace does not depend on the device.  0: it is not.  From 200 shapes of 1 to 16
// rows, or 0.02 to 4 for each of 8 to 64 experts; us, then those of the tensor cores' best form:
//   a row, always (1 x 14336 x 4096 21.0, 22.2; 1 x 4096 x 4096 7.5, 11.6);
//   2 to 4 rows, up to 100 and 80 million multiplications (2 x 13032 x 3768 19.0, 21.2; 3 x 4168 x 7832
//   20.8, 16.8; 4 x 448 x 2376 3.1, 6.2); 8 up to 32 (8 x 1136 x 3376 4.9, 8.1; 8 x 4096 x 4096
//   12.3, 9.9); 16, eight at a time, up to 8 with few outputs (16 x 312 x 1216 4.2, 5.9; 14 x 2552 x 184
//   4.4, 3.8);
//   experts' rows one by one, up to 4 for each, up to 30 and 5000 warps (33 rows, 40 experts,
//   3264 -> 176 8.7, 12.3; 45, 15, 1256 -> 160 4.4, 7.0; 14, 28, 3584 -> 1760 28.9, 25.5; 26, 34,
//   288 -> 888 6.8, 5.1).
int few_rows(const Product& p, const linear_options_t* forced) {
  if (p.kind != LINEAR_FORWARD) return 0;
  if (forced && forced->tile != 0) return forced->tile <= 8 ? forced->tile : 0;
  const double outputs = static_cast<double>(p.n) * static_cast<double>(p.m);
  const double work = 1e-6 * outputs * static_cast<double>(p.k);
  if (p.ragged) return p.n <= 4 * p.groups && work <= 30 && outputs <= 5000 * kFewOuts ? 1 : 0;
  if (p.n <= 1) return 1;
  if (p.n <= 2) return work <= 100 ? 2 : 0;
  if (p.n <= 4) return work <= 80 ? 4 : 0;
  if (p.n <= 8) return work <= 32 ? 8 : 0;
  return p.n <= 16 && p.m <= 512 && work <= 8 ? 8 : 0;
}

// A way of cutting a product, the cycles that it is expected to take, and the SMs that
// it has meanwhile.
struct Form {
  bool pair;
  int tile, split;
  double cycles;
  int64_t ctas;
};
constexpr int kMostForms = 17;

int64_t m_tiles(const Product& p, bool pair) { return pair ? (p.m + 255) / 256 : (p.m + 127) / 128; }

// The forms on the tensor cores.  Cycles, for waves of tiles: a beginning and an end, with what an
// epilogue takes of them by its rows, and blocks of 64 of the sum.  These come in at 60 bytes a
// cycle and SM, and cost something to be issued.  Clusters that share sums meet twice, and send them.
// Fitted to 1200 products of 400 layers (rows 1 to 32768, inputs and outputs 64 to 8192, half of them
// with 8 to 64 experts): 1.2 % over the best form of each in the mean, and half again as long at worst
// (grad_w of 18 experts with 12803 rows, 112 -> 72).
int list_forms(const Product& p, const Machine& machine, Form (&forms)[kMostForms]) {
  const bool weight = p.kind == LINEAR_GRAD_W;
  // of a group, in the mean
  const int64_t k = weight && p.ragged ? (p.k + p.groups - 1) / p.groups : p.k;
  const int64_t n = !weight && p.ragged ? (p.n + p.groups - 1) / p.groups : p.n;
  const double blocks = std::max<double>(1.0, static_cast<double>((k + kLinK - 1) / kLinK));
  const auto cols = [&](int64_t tile) { return static_cast<double>((std::min(tile, n) + 31) / 32 * 32); };
  const auto waves = [](int64_t tiles, int64_t slots) { return static_cast<double>((tiles + slots - 1) / slots); };
  int count = 0;
  const int64_t pairs = machine.sms / 2, pair_tiles = n_tiles(p, 256, false) * m_tiles(p, true);
  forms[count++] = Form{true, 256, 1,
                        360 + waves(pair_tiles, pairs) * (2110 + 19 * cols(256) +
                                                          blocks * std::max(2.6 * cols(256), 520.0)),
                        2 * std::min(pair_tiles, pairs)};
  for (int tile : {32, 64, 128, 256}) {
    if (!valid_form(p.kind, 0, tile, 1)) continue;
    const double c = cols(tile);
    const double block = std::max({1.5 * c, tile > 64 ? 535.0 : 240.0, (kLinABytes + c * 128) / 60.0});
    const int64_t tiles = n_tiles(p, tile, false) * m_tiles(p, false);
    const int64_t most = n_tiles(p, tile, true) * m_tiles(p, false);
    forms[count++] = Form{false, tile, 1, waves(tiles, machine.sms) * (1770 + 19 * c + block * blocks),
                          std::min<int64_t>(tiles, machine.sms)};
    for (int i = 0; i < 3; ++i) {
      const int split = 2 << i;
      if (most > machine.clusters[i] || blocks < 2 * split) continue;
      forms[count++] = Form{false, tile, split,
                            4850 + 36 * c + (68.0 + 9.0 * tiles) * split + block * std::ceil(blocks / split),
                            most * split};
    }
  }
  return count;
}

// The plan of a form that there is.
int plan_of(const Product& p, const Machine& machine, const Form& form, Plan* o) {
  o->pair = form.pair;
  o->tile = form.tile;
  o->split = form.split;
  if (o->tile <= 8) {
    const int64_t units = (p.ragged && o->tile == 1 ? p.n : p.groups) * ((p.m + kFewOuts - 1) / kFewOuts);
    const int64_t blocks = (units * o->split + kFewWarps - 1) / kFewWarps;
    if (blocks > INT_MAX / kFewWarps) return GEMM_ERR_INVALID_VALUE;
    o->m_tiles = o->n_tiles = o->box_rows = 0;
    o->units = static_cast<int>(blocks);
    return GEMM_OK;
  }
  const int64_t most = n_tiles(p, o->tile, true) * m_tiles(p, o->pair);
  // counted in 32 bits, with room for a grid's stride past the last
  if (most > INT_MAX / 4) return GEMM_ERR_INVALID_VALUE;
  o->m_tiles = static_cast<int>(m_tiles(p, o->pair));
  o->n_tiles = p.kind == LINEAR_GRAD_W ? static_cast<int>((p.n + o->tile - 1) / o->tile) : 0;
  // Boxes of 32 rows where a group may end anywhere in a tile, so that a tile loads
  // little more than it has.
  o->box_rows = std::min(p.ragged || p.n <= 64 ? 32 : 128, o->tile);
  o->units = static_cast<int>(o->split > 1 ? most : std::min<int64_t>(o->pair ? machine.sms / 2 : machine.sms, most));
  return GEMM_OK;
}

bool is_forced(const linear_options_t* opt) { return opt && opt->tile != 0; }

int forced_plan(const Product& p, const Machine& machine, const linear_options_t* opt, Plan* o) {
  if (!valid_form(p.kind, opt->cta_pair, opt->tile, opt->split_k)) return GEMM_ERR_INVALID_VALUE;
  return plan_of(p, machine, Form{opt->cta_pair != 0, opt->tile, opt->split_k, 0.0, 0}, o);
}

// The best of `count` forms, of those of `split` CTAs a sum where that is not 0.
const Form* best_of(const Form* forms, int count, int split) {
  const Form* best = nullptr;
  for (int i = 0; i < count; ++i)
    if ((split == 0 || forms[i].split == split) && (!best || forms[i].cycles < best->cycles))
      best = &forms[i];
  return best;
}

// grad_x and grad_w, which run beside each other where the SMs suffice for both (1021 x 1000 x
// 1000: with the form that is best for each alone, 128 CTAs and 128, 17.3 us).  Where memory
// bounds them that does not help.
void choose_both(const Product& x, const Product& w, const Machine& machine, Form* form_x,
                 Form* form_w) {
  Form fx[kMostForms], fw[kMostForms];
  const int nx = list_forms(x, machine, fx), nw = list_forms(w, machine, fw);
  // each weight once, each row of x, dz and their gradients: 16 bits, at 3500 bytes a cycle
  const double weights = static_cast<double>(std::min(x.groups, x.n)) * static_cast<double>(x.m) * static_cast<double>(x.k);
  const double rows = static_cast<double>(x.n) * static_cast<double>(x.m + x.k);
  const double memory = 4.0 * (weights + rows) / 3500.0;
  const Form *best_x = nullptr, *best_w = nullptr;
  double least = 0.0;
  for (int i = 0; i < nx; ++i)
    for (int j = 0; j < nw; ++j) {
      const double cycles = fx[i].ctas + fw[j].ctas <= machine.sms
                                ? std::max({fx[i].cycles, fw[j].cycles, memory}) + 500
                                : fx[i].cycles + fw[j].cycles;
      if (best_x && cycles >= least) continue;
      least = cycles;
      best_x = &fx[i];
      best_w = &fw[j];
    }
  *form_x = *best_x;
  *form_w = *best_w;
}

int make_plans(const Product& x, const Product& w, const Machine& machine,
               const linear_options_t* opt, Plan* plan_x, Plan* plan_w) {
  if (is_forced(opt)) {
    const int rc = forced_plan(x, machine, opt, plan_x);
    return rc != GEMM_OK ? rc : forced_plan(w, machine, opt, plan_w);
  }
  Form fx, fw;
  choose_both(x, w, machine, &fx, &fw);
  const int rc = plan_of(x, machine, fx, plan_x);
  return rc != GEMM_OK ? rc : plan_of(w, machine, fw, plan_w);
}

// A gradient that is asked for alone is cut as it is beside the other one, as far as its bits
// depend on it: by the CTAs that share a sum.  (With the split that is best alone, the bits of
// 64 x 2048 x 2048's grad_x depended on whether grad_w was asked for.  By the estimate, 2 % of
// products take 12 % longer for it in the mean, and 60 % at worst.)
int split_beside(const Product& p, const Machine& machine) {
  Form own, other;
  const bool weight = p.kind == LINEAR_GRAD_W;
  const Product q{weight ? LINEAR_GRAD_X : LINEAR_GRAD_W, p.m, p.k, p.n, p.groups, p.ragged};
  if (weight) choose_both(q, p, machine, &other, &own);
  else choose_both(p, q, machine, &own, &other);
  return own.split;
}

int make_plan(const Product& p, const Machine& machine, const linear_options_t* opt, Plan* o) {
  if (is_forced(opt)) return forced_plan(p, machine, opt, o);
  if (const int rows = few_rows(p, nullptr)) {
    // As many warps for a sum as give each lane 16 bytes of it, and can all run at once
    // (2 x 9112 x 2624: 11.9 us with one, 15.5 with two; 1 x 4096 x 4096: 8.8 with two, 7.5
    // with four).
    const int64_t units = (p.ragged ? p.n : 1) * ((p.m + kFewOuts - 1) / kFewOuts);
    const int64_t warps = machine.sms * kFewWarps * few_blocks(rows, true);
    int split = 1;
    while (split < 8 && 2 * split * units <= warps && split * 256 < p.k) split *= 2;
    return plan_of(p, machine, Form{false, rows, split, 0.0, 0}, o);
  }
  Form forms[kMostForms];
  const int count = list_forms(p, machine, forms);
  const int split = p.kind == LINEAR_FORWARD ? 0 : split_beside(p, machine);
  return plan_of(p, machine, *best_of(forms, count, split), o);
}

// ------------------------------------------------------------------ launches
struct Maps {
  CUtensorMap a, b;
};

// A matrix of `rows` rows of `cols` as two or three dimensions (matrices of it).
int encode(EncodeTiledFn fn, CUtensorMap* map, const void* ptr, int64_t cols, int64_t rows,
           int64_t ld, int64_t matrices, uint32_t box_rows, int rank) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(matrices)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2,
                                 static_cast<cuuint64_t>(ld) * 2 * (matrices > 1 ? rows : 1)};
  const cuuint32_t box[3] = {kLinK, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, rank, const_cast<void*>(ptr), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

template <typename T, int kProduct>
int launch_as(const Maps& m, LinearParams p, const Plan& plan, int device, cudaStream_t s) {
  const uint32_t fixed = linear_fixed_bytes(p.groups);
  const uint32_t block = plan.pair ? kLinPairStage : kLinABytes + plan.tile * (kLinK * 2);
  const int blocks = plan.pair || plan.tile > 64 ? 1 : 2;
  const uint32_t stage = blocks * block;
  p.stages = std::min<int>((kLinSmemLimit - fixed) / stage, kLinMaxStages / blocks);
  const size_t smem = fixed + p.stages * stage;
  const auto go = [&](auto kernel, std::atomic<uint64_t>& granted, unsigned ctas, unsigned cluster) {
    if (!grant_smem(kernel, kLinSmemLimit, device, granted)) return static_cast<int>(GEMM_ERR_CUDA);
    return launch_pdl(kernel, dim3(ctas), dim3(kLinThreads), smem, s, cluster, m.a, m.b, p);
  };
  static std::atomic<uint64_t> granted[5];
  if (plan.pair) return go(linear_pair<T, kProduct>, granted[0], 2 * plan.units, 2);
  if (plan.split > 1)
    return blocks == 2
               ? go(linear_tc<T, kProduct, true, 2>, granted[1], plan.units * plan.split, plan.split)
               : go(linear_tc<T, kProduct, true, 1>, granted[2], plan.units * plan.split, plan.split);
  return blocks == 2 ? go(linear_tc<T, kProduct, false, 2>, granted[3], plan.units, 1)
                     : go(linear_tc<T, kProduct, false, 1>, granted[4], plan.units, 1);
}

template <typename T, int kRows>
int launch_few(const FewParams& f, const LinearParams& p, bool aligned, int blocks,
               cudaStream_t s) {
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kFewThreads), 0, s, 1u, f, p);
  };
  return aligned ? go(linear_few<T, kRows, true>) : go(linear_few<T, kRows, false>);
}

// The forward product of few rows: x and w as the caller has them.
int launch_few(const Plan& plan, const Rows& w, const Rows& x, LinearParams p, int type,
               cudaStream_t s) {
  const FewParams f{static_cast<const uint16_t*>(x.ptr), static_cast<const uint16_t*>(w.ptr), x.ld,
                    w.ld};
  p.n = static_cast<int32_t>(w.rows / p.groups);
  p.k = static_cast<int32_t>(w.cols);
  p.split = plan.split;
  const bool aligned = loads_as_is(x) && loads_as_is(w) && p.k % 8 == 0;
  const auto by_type = [&](auto t) {
    using T = decltype(t);
    switch (plan.tile) {
      case 1: return launch_few<T, 1>(f, p, aligned, plan.units, s);
      case 2: return launch_few<T, 2>(f, p, aligned, plan.units, s);
      case 4: return launch_few<T, 4>(f, p, aligned, plan.units, s);
      default: return launch_few<T, 8>(f, p, aligned, plan.units, s);
    }
  };
  return type == MOE_F16 ? by_type(__half{}) : by_type(__nv_bfloat16{});
}

// One product of operands that the tensor maps take as they are: `a` is that of M, w or
// (grad_w) x, and `b` that of N, x or dz.
int launch(const Product& pr, const Plan& plan, const Rows& a, const Rows& b, LinearParams p,
           int type, const linear_options_t* opt, int device, cudaStream_t s) {
  int rc = GEMM_OK;
  const bool weight = pr.kind == LINEAR_GRAD_W;
  p.n = static_cast<int32_t>(pr.m);
  p.m = weight ? static_cast<int32_t>(pr.n) : 0;
  p.k = static_cast<int32_t>(pr.k);
  p.groups = static_cast<int32_t>(pr.groups);
  p.tile = plan.tile;
  while (1 << p.tile_shift < p.tile) ++p.tile_shift;
  p.m_tiles = plan.m_tiles;
  p.n_tiles = plan.n_tiles;
  p.box_rows = plan.box_rows;
  p.split = plan.split;
  p.inject = opt ? opt->inject : 0;
  p.timeout_ns = opt && opt->timeout_ns
                     ? opt->timeout_ns
                     : kTimeoutNs + kTimeoutNsPerBlock * static_cast<uint64_t>(pr.k / kLinK);
  p.error_word = error_index(s);
  Maps m;
  std::memset(&m, 0, sizeof(m));
  if (pr.k > 0) {
    EncodeTiledFn fn = nullptr;
    if ((rc = get_encoder(&fn)) != GEMM_OK) return rc;
    const int64_t matrices = weight ? 1 : pr.groups;
    if ((rc = encode(fn, &m.a, a.ptr, a.cols, a.rows / matrices, a.ld, matrices,
                     pr.kind == LINEAR_FORWARD ? kLinM : 64, 3)) != GEMM_OK ||
        (rc = encode(fn, &m.b, b.ptr, b.cols, b.rows, b.ld, 1, weight ? 64 : plan.box_rows, 2)) !=
            GEMM_OK)
      return rc;
  }
  const auto by_type = [&](auto t) {
    using T = decltype(t);
    switch (pr.kind) {
      case LINEAR_FORWARD: return launch_as<T, LINEAR_FORWARD>(m, p, plan, device, s);
      case LINEAR_GRAD_X: return launch_as<T, LINEAR_GRAD_X>(m, p, plan, device, s);
      default: return launch_as<T, LINEAR_GRAD_W>(m, p, plan, device, s);
    }
  };
  return type == MOE_F16 ? by_type(__half{}) : by_type(__nv_bfloat16{});
}

// ------------------------------------------------------------------ workspaces
// Pieces of a workspace, one after the other, each on a 16-byte boundary.
struct Pieces {
  uint64_t bytes = 0;
  uint64_t add(uint64_t n) {
    const uint64_t at = bytes;
    bytes += (n + 15) & ~uint64_t{15};
    return at;
  }
};
uint64_t copy_bytes(const Rows& r) { return static_cast<uint64_t>(r.rows) * copy_ld(r.cols) * 2; }

struct ForwardSpace {
  bool copy_x, copy_w;
  uint64_t x, w, bytes;
};
ForwardSpace forward_space(const linear_t* l, bool few) {
  Pieces p;
  ForwardSpace f{};
  const bool sums = !few && l->rows > 0 && l->out > 0 && l->in > 0;
  f.copy_x = sums && !loads_as_is(x_rows(l));
  f.copy_w = sums && !loads_as_is(w_rows(l));
  if (f.copy_x) f.x = p.add(copy_bytes(x_rows(l)));
  if (f.copy_w) f.w = p.add(copy_bytes(w_rows(l)));
  f.bytes = p.bytes;
  return f;
}

struct BackwardSpace {
  bool copy_x, copy_w, dz, strips;
  uint64_t x, w, z, sums, bytes;
  int strip_rows;
};
BackwardSpace backward_space(const linear_t* l, bool grad_x, bool grad_w, bool grad_bias,
                             const Rows& grad) {
  Pieces p;
  BackwardSpace b{};
  const bool live = l->rows > 0 && l->out > 0;
  const bool for_x = live && grad_x && l->in > 0, for_w = live && grad_w && l->in > 0;
  b.copy_w = for_x && !loads_as_is(w_rows(l));
  b.copy_x = for_w && !loads_as_is(x_rows(l));
  b.dz = (for_x || for_w) && (l->activation != LINEAR_NONE || !loads_as_is(grad));
  b.strips = live && grad_bias;
  b.strip_rows = strip_rows_for(l->rows, l->out);
  if (b.copy_w) b.w = p.add(copy_bytes(w_rows(l)));
  if (b.copy_x) b.x = p.add(copy_bytes(x_rows(l)));
  if (b.dz) b.z = p.add(copy_bytes(grad));
  if (b.strips)
    b.sums = p.add((l->rows / b.strip_rows + groups_of(l)) * strip_ld(l->out) * 4);
  b.bytes = p.bytes;
  return b;
}

int check_workspace(const void* workspace, uint64_t bytes, uint64_t needed) {
  if (needed == 0) return GEMM_OK;
  if (!workspace || bytes < needed) return GEMM_ERR_INVALID_VALUE;
  return aligned_to(workspace, 16) ? GEMM_OK : GEMM_ERR_MISALIGNED;
}

// Has rows copied to `at` of the workspace, and takes them from there.
void copied(Rows* r, PrepareRows* p, int which, void* workspace, uint64_t at) {
  p->from[which] = *r;
  p->to[which] = static_cast<uint8_t*>(workspace) + at;
  r->ptr = p->to[which];
  r->ld = copy_ld(r->cols);
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" int linear_forward_workspace(const linear_t* layer, const linear_options_t* opt,
                                        uint64_t* bytes) {
  int rc = check_layer(layer);
  if (rc != GEMM_OK) return rc;
  if ((rc = check_options(opt)) != GEMM_OK) return rc;
  if (!bytes) return GEMM_ERR_INVALID_VALUE;
  *bytes = forward_space(layer, few_rows(forward_of(layer), opt) > 0).bytes;
  return GEMM_OK;
}

extern "C" int linear_backward_workspace(const void* grad_x, const void* grad_w,
                                         const void* grad_bias, const linear_t* layer,
                                         const void* grad_out, int64_t ldg, uint64_t* bytes) {
  const int rc = check_layer(layer);
  if (rc != GEMM_OK) return rc;
  if (!bytes) return GEMM_ERR_INVALID_VALUE;
  *bytes = backward_space(layer, grad_x != nullptr, grad_w != nullptr, grad_bias != nullptr,
                          by_out(layer, grad_out, ldg)).bytes;
  return GEMM_OK;
}

extern "C" int linear_forward(void* out, void* preact, const linear_t* layer, const void* bias,
                              const void* residual, int64_t ldr, void* workspace,
                              uint64_t workspace_bytes, const linear_options_t* opt, void* stream) {
  int rc = check_layer(layer);
  if (rc != GEMM_OK) return rc;
  if ((rc = check_options(opt)) != GEMM_OK) return rc;
  const Rows result = by_out(layer, out, layer->out);
  Rows x = x_rows(layer), w = w_rows(layer);
  const Rows res = by_out(layer, residual, ldr);
  if (residual && layer->routing) return GEMM_ERR_INVALID_VALUE;
  for (const Rows* r : {&x, &w})
    if ((rc = check_rows(*r)) != GEMM_OK) return rc;
  if (residual && (rc = check_rows(res)) != GEMM_OK) return rc;
  if (!aligned_to(preact, 2) || !aligned_to(bias, 2)) return GEMM_ERR_MISALIGNED;
  const Product pr = forward_of(layer);
  const ForwardSpace space = forward_space(layer, few_rows(pr, opt) > 0);
  if ((rc = check_workspace(workspace, workspace_bytes, space.bytes)) != GEMM_OK) return rc;
  if (layer->rows == 0 || layer->out == 0) return GEMM_OK;
  if ((rc = check_rows(result)) != GEMM_OK) return rc;
  const int groups = groups_of(layer);
  if (any_overlap({{out, bytes_of(result), true},
                   {preact, bytes_of(result), true},
                   {space.bytes ? workspace : nullptr, space.bytes, true},
                   {bias, static_cast<uint64_t>(groups) * layer->out * 2, false},
                   reads(x), reads(w), reads(res)},
                  layer->routing))
    return GEMM_ERR_INVALID_VALUE;
  int sms = 0, device = 0;
  if ((rc = require_device(&sms, &device)) != GEMM_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LinearParams p;
  std::memset(&p, 0, sizeof(p));
  p.out = static_cast<uint16_t*>(out);
  p.preact = static_cast<uint16_t*>(preact);
  p.bias = static_cast<const uint16_t*>(bias);
  p.residual = static_cast<const uint16_t*>(residual);
  p.ldr = res.ld;
  p.offsets = offsets_of(layer);
  p.rows = static_cast<int32_t>(layer->rows);
  p.activation = layer->activation;
  p.groups = groups;
  Machine machine;
  Plan plan;
  if ((rc = machine_of(sms, device, &machine)) != GEMM_OK ||
      (rc = make_plan(pr, machine, opt, &plan)) != GEMM_OK)
    return rc;
  if (plan.tile <= 8) return launch_few(plan, w, x, p, layer->type, s);
  PrepareRows prepare{};
  prepare.type = layer->type;
  if (space.copy_x) copied(&x, &prepare, 0, workspace, space.x);
  if (space.copy_w) copied(&w, &prepare, 1, workspace, space.w);
  if ((rc = prepare_rows(prepare, s)) != GEMM_OK) return rc;
  return launch(pr, plan, w, x, p, layer->type, opt, device, s);
}

extern "C" int linear_backward(void* grad_x, void* grad_w, void* grad_bias, const linear_t* layer,
                               const void* grad_out, int64_t ldg, const void* preact,
                               void* workspace, uint64_t workspace_bytes,
                               const linear_options_t* opt, void* stream) {
  int rc = check_layer(layer);
  if (rc != GEMM_OK) return rc;
  if ((rc = check_options(opt)) != GEMM_OK) return rc;
  const int groups = groups_of(layer);
  Rows x = x_rows(layer), w = w_rows(layer), dz = by_out(layer, grad_out, ldg);
  const Rows z = by_out(layer, preact, layer->out);
  const Rows to_x = matrix_of(grad_x, layer->rows, layer->in, layer->in);
  const Rows to_w = matrix_of(grad_w, groups * layer->out, layer->in, layer->in);
  const uint64_t bias_bytes = static_cast<uint64_t>(groups) * layer->out * 2;
  if ((rc = check_rows(dz)) != GEMM_OK) return rc;
  if (layer->activation != LINEAR_NONE && (rc = check_rows(z)) != GEMM_OK) return rc;
  if (grad_w && (rc = check_rows(x)) != GEMM_OK) return rc;
  if (grad_x && (rc = check_rows(w)) != GEMM_OK) return rc;
  if (!aligned_to(grad_x, 2) || !aligned_to(grad_w, 2) || !aligned_to(grad_bias, 2))
    return GEMM_ERR_MISALIGNED;
  const BackwardSpace space =
      backward_space(layer, grad_x != nullptr, grad_w != nullptr, grad_bias != nullptr, dz);
  if ((rc = check_workspace(workspace, workspace_bytes, space.bytes)) != GEMM_OK) return rc;
  if (any_overlap({{grad_x, bytes_of(to_x), true},
                   {grad_w, bytes_of(to_w), true},
                   {grad_bias, bias_bytes, true},
                   {space.bytes ? workspace : nullptr, space.bytes, true},
                   {grad_w ? x.ptr : nullptr, bytes_of(x), false},
                   {grad_x ? w.ptr : nullptr, bytes_of(w), false},
                   {layer->activation != LINEAR_NONE ? preact : nullptr, bytes_of(z), false},
                   reads(dz)},
                  layer->routing))
    return GEMM_ERR_INVALID_VALUE;
  const bool for_x = grad_x && bytes_of(to_x) > 0, for_w = grad_w && bytes_of(to_w) > 0,
             for_bias = grad_bias && bias_bytes > 0;
  if (!for_x && !for_w && !for_bias) return GEMM_OK;
  int sms = 0, device = 0;
  if ((rc = require_device(&sms, &device)) != GEMM_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Machine machine;
  if ((rc = machine_of(sms, device, &machine)) != GEMM_OK) return rc;

  LinearParams p;
  std::memset(&p, 0, sizeof(p));
  p.offsets = offsets_of(layer);
  p.rows = static_cast<int32_t>(layer->rows);
  p.strip_rows = space.strip_rows;
  const auto at = [&](uint64_t offset) { return static_cast<uint8_t*>(workspace) + offset; };
  float* const strips = space.strips ? reinterpret_cast<float*>(at(space.sums)) : nullptr;
  PrepareRows prepare{};
  prepare.type = layer->type;
  if (space.dz || space.strips) {
    prepare.grad = dz;
    prepare.preact = layer->activation == LINEAR_NONE ? nullptr : preact;
    prepare.dz = space.dz ? at(space.z) : nullptr;
    prepare.strips = strips;
    prepare.offsets = p.offsets;
    prepare.groups = groups;
    prepare.strip_rows = space.strip_rows;
    prepare.activation = layer->activation;
    if (space.dz) {
      dz.ptr = prepare.dz;
      dz.ld = copy_ld(dz.cols);
    }
  }
  if (space.copy_w) copied(&w, &prepare, 0, workspace, space.w);
  if (space.copy_x) copied(&x, &prepare, 1, workspace, space.x);
  const Product pr_x = product_of(LINEAR_GRAD_X, layer->rows, layer->in, layer->out, groups,
                                  p.offsets != nullptr);
  const Product pr_w = product_of(LINEAR_GRAD_W, layer->rows, layer->in, layer->out, groups,
                                  p.offsets != nullptr);
  Plan plan_x, plan_w;
  if (for_x && for_w) rc = make_plans(pr_x, pr_w, machine, opt, &plan_x, &plan_w);
  else if (for_x) rc = make_plan(pr_x, machine, opt, &plan_x);
  else if (for_w) rc = make_plan(pr_w, machine, opt, &plan_w);
  if (rc != GEMM_OK || (rc = prepare_rows(prepare, s)) != GEMM_OK) return rc;
  // Between the launches of the two products there is no other (see launch_pdl).
  if (for_x) {
    LinearParams px = p;
    px.out = static_cast<uint16_t*>(grad_x);
    px.overlap = for_w ? kOverlapFirst : kOverlapNone;
    if ((rc = launch(pr_x, plan_x, w, dz, px, layer->type, opt, device, s)) != GEMM_OK) return rc;
  }
  p.grad_bias = static_cast<uint16_t*>(grad_bias);
  if (for_w) {
    p.out = static_cast<uint16_t*>(grad_w);
    p.strips = for_bias ? strips : nullptr;
    p.overlap = for_x ? kOverlapSecond : kOverlapNone;
    rc = launch(pr_w, plan_w, x, dz, p, layer->type, opt, device, s);
    if (rc != GEMM_OK || strips) return rc;
  }
  if (!for_bias) return GEMM_OK;
  // Without grad_w, or without rows: then there are no strips either.
  p.m = static_cast<int32_t>(layer->out);
  p.groups = groups;
  p.strips = strips;
  return sum_strips(p, layer->type, sms, s);
}

extern "C" int linear_query_config(int product, int64_t rows, int64_t in, int64_t out, int experts,
                                   linear_config_t* config) {
  if (!config || product < LINEAR_FORWARD || product > LINEAR_GRAD_W_OF_BOTH || rows < 1 || in < 1 ||
      out < 1 || rows > LINEAR_MAX_ROWS || in > LINEAR_MAX_COLS || out > LINEAR_MAX_COLS ||
      experts < 0 || experts > MOE_MAX_EXPERTS || std::max(experts, 1) * out > INT_MAX)
    return GEMM_ERR_INVALID_VALUE;
  Machine machine{152, {76, 36, 15}};
  int sms = 0, device = 0, rc = GEMM_OK;
  if (require_device(&sms, &device) != GEMM_OK) cudaGetLastError();
  else if ((rc = machine_of(sms, device, &machine)) != GEMM_OK) return rc;
  const auto of = [&](int kind) {
    return product_of(kind, rows, in, out, std::max(experts, 1), experts > 0);
  };
  Plan plan, beside;
  if (product == LINEAR_GRAD_X_OF_BOTH)
    rc = make_plans(of(LINEAR_GRAD_X), of(LINEAR_GRAD_W), machine, nullptr, &plan, &beside);
  else if (product == LINEAR_GRAD_W_OF_BOTH)
    rc = make_plans(of(LINEAR_GRAD_X), of(LINEAR_GRAD_W), machine, nullptr, &beside, &plan);
  else
    rc = make_plan(of(product), machine, nullptr, &plan);
  if (rc != GEMM_OK) return rc;
  *config = linear_config_t{plan.pair ? 1 : 0, plan.tile, plan.split,
                            plan.units * (plan.pair ? 2 : plan.tile <= 8 ? 1 : plan.split)};
  return GEMM_OK;
}

extern "C" int linear_get_device_error(void* stream, uint32_t* raw) {
  const int rc = require_device(nullptr);
  if (rc != GEMM_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  const uint32_t zero = 0;
  const size_t off = static_cast<size_t>(error_index(s)) * sizeof(uint32_t);
  if (cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&word, g_linear_error, sizeof(word), off, cudaMemcpyDeviceToHost,
                                s) != cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_linear_error, &zero, sizeof(zero), off, cudaMemcpyHostToDevice, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (raw) *raw = word;
  return static_cast<int>(word & 0xffu);
}
