// Python binding of moe_fp4.h and linear.h: checks and marshals torch tensors, allocates
// outputs, and calls the C functions on the current (or a given) stream.  It
// is compiled because the calls it makes are a few microseconds long on the
// GPU: marshalled from Python, a call cost the host 7 to 11 us; compiled, 2.6 to
// 4.3, of which a launch is 1.5 and an allocation 0.6.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>

#include <memory>
#include <optional>
#include <string>
#include <tuple>

#include "moe_fp4.h"

namespace {

[[noreturn]] void value_error(const std::string& what) { throw py::value_error(what); }
[[noreturn]] void type_error(const std::string& what) { throw py::type_error(what); }

// A C function's status, as the exception the fp16 binding raises.
void check(int status, const char* name) {
  if (status == GEMM_OK) return;
  const py::object error =
      py::module_::import("multistage_smem_pipeline_gb300.binding").attr("GemmError");
  const py::object value = error(status, name);
  PyErr_SetObject(error.ptr(), value.ptr());
  throw py::error_already_set();
}

// The stream a call runs on, current meanwhile together with its device: what is
// allocated then belongs to that stream, and is not memory that work queued on
// another one may still be using.
class On {
 public:
  On(at::Device device, const py::object& stream) {
    if (stream.is_none()) {
      device_.emplace(device);
      handle_ = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    } else {
      handle_ = reinterpret_cast<cudaStream_t>(stream.attr("cuda_stream").cast<uintptr_t>());
      stream_.emplace(c10::cuda::getStreamFromExternal(handle_, device.index()));
    }
  }
  void* stream() const { return handle_; }

 private:
  std::optional<c10::cuda::CUDAGuard> device_;
  std::optional<c10::cuda::CUDAStreamGuard> stream_;
  cudaStream_t handle_ = nullptr;
};

int type_of(at::ScalarType t, const char* what) {
  if (t == at::kHalf) return MOE_F16;
  if (t == at::kBFloat16) return MOE_BF16;
  type_error(std::string(what) + " must be float16 or bfloat16");
}

at::ScalarType dtype_of(const py::object& dtype) {
  if (dtype.is_none()) return at::kHalf;
  if (!THPDtype_Check(dtype.ptr())) type_error("dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(dtype.ptr())->scalar_type;
}

int format_of(const std::string& name) {
  if (name == "nvfp4") return FP4_NV;
  if (name == "mxfp4") return FP4_MX;
  value_error("unknown format '" + name + "'");
}
const char* format_name(int format) { return format == FP4_NV ? "nvfp4" : "mxfp4"; }

// x is a CUDA matrix of a supported type with contiguous rows; its type number.
int matrix(const at::Tensor& x, const char* what) {
  const int type = type_of(x.scalar_type(), what);
  const std::string name(what);
  if (x.dim() != 2) value_error(name + " must be a 2-D CUDA tensor");
  if (x.size(1) > 1 && x.stride(1) != 1) value_error(name + "'s rows must be contiguous");
  if (x.size(0) > 1 && x.stride(0) < x.size(1))  // an expanded row, or windows over one
    value_error(name + "'s rows must not overlap");
  if (!x.is_cuda()) value_error(name + " must be a 2-D CUDA tensor");
  return type;
}

// Elements between rows (a tensor of one row may report any stride).
int64_t row_stride(const at::Tensor& x) { return x.size(0) > 1 ? x.stride(0) : x.size(1); }

// at::empty for the GPU, without the dispatcher's part of its time.
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, at::Device device) {
  return at::detail::empty_cuda(sizes, type, device, std::nullopt);
}

using Out = std::optional<at::Tensor>;

at::Tensor output(const Out& out, int64_t rows, int64_t cols, at::ScalarType type,
                  at::Device device) {
  if (!out) return fresh({rows, cols}, type, device);
  if (out->scalar_type() != type || out->dim() != 2 || out->size(0) != rows ||
      out->size(1) != cols || !out->is_contiguous() || out->device() != device)
    value_error("out must be a contiguous " + std::to_string(rows) + " x " +
                std::to_string(cols) + " tensor of the right type on the inputs' device");
  return *out;
}

// Part of a buffer from element `first` on, contiguous: a tensor over the same
// storage, made directly (through the dispatcher a view costs the host 1 to 5 us,
// which is as long as some of the kernels).
at::Tensor part(const at::Tensor& buffer, int64_t first, at::IntArrayRef sizes) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::TensorImpl::VIEW, c10::Storage(buffer.storage()), buffer.key_set(), buffer.dtype());
  c10::TensorImpl* const impl = t.unsafeGetTensorImpl();
  impl->set_version_counter(buffer.unsafeGetTensorImpl()->version_counter());
  impl->set_storage_offset(first);
  impl->set_sizes_contiguous(sizes);
  return t;
}

// ------------------------------------------------------------------ Routing
struct Routing {
  at::Tensor ids, buffer;     // buffer: the two arrays of moe_sort, in one piece
  at::Tensor offsets, rows;   // made from it when they are asked for
  moe_routing_t c{};

  int64_t slots() const { return c.tokens * c.top_k; }
  int64_t head() const { return (c.experts + 4) & ~int64_t{3}; }      // offsets, to 16 bytes
  at::Device device() const { return ids.device(); }

  void describe(int64_t experts) {
    c.tokens = ids.size(0);
    c.top_k = static_cast<int32_t>(ids.size(1));
    c.experts = static_cast<int32_t>(experts);
    c.ids = static_cast<const int32_t*>(ids.data_ptr());
  }

  const at::Tensor& get_offsets() {
    if (!offsets.defined()) offsets = part(buffer, 0, {c.experts + 1});
    return offsets;
  }
  const at::Tensor& get_rows() {
    if (!rows.defined()) rows = part(buffer, head(), {c.tokens, c.top_k});
    return rows;
  }
};
using RoutingPtr = std::shared_ptr<Routing>;

// A routing's arrays are where the tensor is that they speak of.
void same_device(const at::Device& device, const RoutingPtr& r, const char* what) {
  if (r && r->device() != device)
    value_error(std::string(what) + " and the routing are on different devices");
}

RoutingPtr given_routing(const at::Tensor& offsets, const at::Tensor& rows,
                         const at::Tensor& ids) {
  for (const at::Tensor* t : {&offsets, &rows, &ids})
    if (t->scalar_type() != at::kInt || !t->is_cuda() || !t->is_contiguous() ||
        t->device() != ids.device())
      value_error("offsets, rows and ids must be contiguous int32 CUDA tensors on one device");
  if (ids.dim() != 2 || rows.sizes() != ids.sizes() || offsets.dim() != 1 || offsets.numel() < 2)
    value_error("ids and rows must be tokens x top_k, and offsets experts + 1");
  auto r = std::make_shared<Routing>();
  r->ids = ids;
  r->offsets = offsets;
  r->rows = rows;
  r->describe(offsets.numel() - 1);
  r->c.offsets = static_cast<const int32_t*>(offsets.data_ptr());
  r->c.rows = static_cast<const int32_t*>(rows.data_ptr());
  return r;
}

RoutingPtr sort(const at::Tensor& ids, int64_t experts, const py::object& stream) {
  if (ids.scalar_type() != at::kInt) type_error("ids must be int32");
  if (ids.dim() != 2 || !ids.is_cuda() || !ids.is_contiguous())
    value_error("ids must be a contiguous 2-D CUDA tensor (tokens x top_k)");
  if (experts < 1 || experts > MOE_MAX_EXPERTS || ids.size(1) < 1 || ids.size(1) > MOE_MAX_TOP_K)
    value_error("1 to " + std::to_string(MOE_MAX_EXPERTS) + " experts and 1 to " +
                std::to_string(MOE_MAX_TOP_K) + " slots are supported");
  const On on(ids.device(), stream);
  auto r = std::make_shared<Routing>();
  r->ids = ids;
  r->describe(experts);
  r->buffer = fresh({r->head() + r->slots()}, at::kInt, ids.device());
  int32_t* const at = static_cast<int32_t*>(r->buffer.data_ptr());
  r->c.offsets = at;
  r->c.rows = at + r->head();
  check(moe_sort(at, at + r->head(), r->c.ids, r->c.tokens, r->c.top_k, r->c.experts, on.stream()),
        "moe_sort");
  return r;
}

at::Tensor pairs_of(const Routing& r, const py::object& stream) {
  const On on(r.device(), stream);
  const at::Tensor pairs = fresh({r.slots()}, at::kInt, r.device());
  check(moe_pairs(static_cast<int32_t*>(pairs.data_ptr()), &r.c, on.stream()), "moe_pairs");
  return pairs;
}

// ------------------------------------------------------------------ Fp4Matrix
struct Fp4Matrix {
  at::Tensor buffer;           // scales, then codes, in one piece
  at::Tensor codes, scales;    // made from it when they are asked for
  RoutingPtr routing;
  int64_t pitch = 0, tiles = 0, chunks = 0;
  at::Device device{at::kCUDA};
  fp4_matrix_t c{};

  // Everything but the pointers.
  void describe(int64_t rows, int64_t cols, int format, int64_t exponent,
                std::optional<int64_t> group_rows, const RoutingPtr& r) {
    if (exponent != static_cast<int32_t>(exponent))  // the C functions check the rest
      value_error("exponent " + std::to_string(exponent) + " is out of range");
    if (rows > INT32_MAX) value_error(std::to_string(rows) + " rows are too many");
    c.rows = rows;
    c.cols = cols;
    c.format = format;
    c.exponent = static_cast<int32_t>(exponent);
    pitch = (cols + 31) / 32 * 16;
    chunks = (cols + 255) / 256 * (format == FP4_NV ? 4 : 2);
    routing = r;
    if (r) {
      if (group_rows || rows != r->slots())
        value_error("a matrix in expert order has a row per slot and no group_rows");
      c.groups = r->c.experts;
      c.offsets = r->c.offsets;
      tiles = rows / 128 + c.groups;
      return;
    }
    const int64_t g = group_rows.value_or(rows);
    if (g < 0 || (g ? rows % g : rows) != 0)
      value_error(std::to_string(rows) + " rows are not whole groups of " + std::to_string(g));
    c.groups = g ? static_cast<int32_t>(std::max<int64_t>(rows / g, 1)) : 1;
    c.group_rows = rows ? g : 0;  // no rows are whole groups of any size
    tiles = c.groups * ((c.group_rows + 127) / 128);
  }

  const at::Tensor& get_scales() {
    if (!scales.defined())
      scales = part(buffer, 0, {tiles, chunks, 512});
    return scales;
  }
  const at::Tensor& get_codes() {
    if (!codes.defined())
      codes = part(buffer, tiles * chunks * 512, {c.rows, pitch});
    return codes;
  }
};
using MatrixPtr = std::shared_ptr<Fp4Matrix>;

MatrixPtr given_matrix(const at::Tensor& codes, const at::Tensor& scales, int64_t cols,
                       const std::string& format, int64_t exponent,
                       std::optional<int64_t> group_rows, const RoutingPtr& routing) {
  const int fmt = format_of(format);
  if (codes.scalar_type() != at::kByte || scales.scalar_type() != at::kByte)
    type_error("codes and scales must be uint8");
  if (!codes.is_cuda() || !scales.is_cuda() || codes.device() != scales.device())
    value_error("codes and scales must be CUDA tensors on one device");
  if (!codes.is_contiguous() || !scales.is_contiguous())
    value_error("codes and scales must be contiguous");
  same_device(codes.device(), routing, "codes");
  if (codes.dim() != 2 || cols < 0 || cols > FP4_MAX_COLS)
    value_error("codes must be a matrix of 0 to " + std::to_string(FP4_MAX_COLS) + " columns");
  auto m = std::make_shared<Fp4Matrix>();
  m->describe(codes.size(0), cols, fmt, exponent, group_rows, routing);
  if (codes.size(1) != m->pitch)
    value_error("codes must have " + std::to_string(m->pitch) + " bytes a row, got " +
                std::to_string(codes.size(1)));
  if (scales.numel() < m->tiles * m->chunks * 512)
    value_error("scales must have " + std::to_string(m->tiles * m->chunks * 512) +
                " bytes, got " + std::to_string(scales.numel()));
  m->codes = codes;
  m->scales = scales;
  m->device = codes.device();
  m->c.codes = codes.data_ptr();
  m->c.scales = scales.data_ptr();
  return m;
}

MatrixPtr quantize(const at::Tensor& x, const std::string& format, int64_t exponent,
                   std::optional<int64_t> group_rows, const RoutingPtr& routing,
                   const MatrixPtr& out, const py::object& stream) {
  const int type = matrix(x, "x");
  const int fmt = format_of(format);
  int64_t rows = x.size(0);
  const int64_t cols = x.size(1);
  if (routing) {
    if (rows != routing->c.tokens)
      value_error("x has " + std::to_string(rows) + " rows, the routing " +
                  std::to_string(routing->c.tokens) + " tokens");
    same_device(x.device(), routing, "x");
    rows = routing->slots();
  }
  MatrixPtr m = out;
  if (!m) {
    m = std::make_shared<Fp4Matrix>();
    m->describe(rows, cols, fmt, exponent, group_rows, routing);
  }
  const On on(x.device(), stream);
  if (!out) {
    const int64_t scales = m->tiles * m->chunks * 512;
    m->buffer = fresh({scales + rows * m->pitch}, at::kByte, x.device());
    m->device = x.device();
    m->c.scales = m->buffer.data_ptr();
    m->c.codes = static_cast<uint8_t*>(m->buffer.data_ptr()) + scales;
  } else if (m->c.rows != rows || m->c.cols != cols || m->c.format != fmt ||
             m->c.exponent != exponent || m->routing != routing || m->device != x.device() ||
             (group_rows && m->c.group_rows != *group_rows)) {
    value_error("out does not fit x, the format or the groups");
  }
  check(fp4_quantize(&m->c, x.data_ptr(), row_stride(x), type, routing ? &routing->c : nullptr,
                     on.stream()),
        "fp4_quantize");
  return m;
}

at::Tensor dequantize(const Fp4Matrix& q, const py::object& dtype, const Out& out,
                      const py::object& stream) {
  const at::ScalarType t = dtype_of(dtype);
  const int type = type_of(t, "dtype");
  const On on(q.device, stream);
  const at::Tensor y = output(out, q.c.rows, q.c.cols, t, q.device);
  check(fp4_dequantize(y.data_ptr(), type, &q.c, on.stream()), "fp4_dequantize");
  return y;
}

at::Tensor gemm(const Fp4Matrix& a, const Fp4Matrix& b, double alpha, const py::object& dtype,
                const Out& out, const py::object& stream, uint64_t timeout_ns, int inject) {
  const at::ScalarType t = dtype_of(dtype);
  const int type = type_of(t, "dtype");
  if (a.device != b.device) value_error("a and b are on different devices");
  const On on(a.device, stream);
  const at::Tensor d = output(out, a.c.rows, b.c.group_rows, t, a.device);
  fp4_matrix_t rows = a.c;
  if (rows.rows == 0 && !rows.offsets) rows.groups = b.c.groups;  // ... and any number of them
  check(fp4_gemm_tn_ex(d.data_ptr(), type, &rows, &b.c, static_cast<float>(alpha), timeout_ns, inject,
                       on.stream()),
        "fp4_gemm_tn");
  return d;
}

// On the stream's own device; other threads of the interpreter run meanwhile.
py::tuple device_error(const py::object& stream, int (*read)(void*, uint32_t*)) {
  std::optional<c10::cuda::CUDAGuard> device;
  if (!stream.is_none() && py::hasattr(stream, "device"))
    device.emplace(stream.attr("device").cast<at::Device>());
  void* const s = stream.is_none()
                      ? static_cast<void*>(c10::cuda::getCurrentCUDAStream().stream())
                      : reinterpret_cast<void*>(stream.attr("cuda_stream").cast<uintptr_t>());
  uint32_t raw = 0;
  int status = 0;
  {
    const py::gil_scoped_release released;
    status = read(s, &raw);
  }
  return py::make_tuple(status, raw);
}

int64_t scale_bytes(int64_t rows, int64_t cols, const std::string& format, int groups,
                    bool by_offsets) {
  uint64_t n = 0;
  check(fp4_scale_bytes(rows, cols, format_of(format), groups, by_offsets, &n), "fp4_scale_bytes");
  return static_cast<int64_t>(n);
}

py::dict query_config(int64_t rows, int64_t n, int64_t cols, const std::string& format, int groups,
                      bool by_offsets) {
  fp4_config_t c{};
  check(fp4_query_config(rows, n, cols, format_of(format), groups, by_offsets, &c),
        "fp4_query_config");
  py::dict d;
  d["cta_pair"] = c.cta_pair;
  d["split_k"] = c.split_k;
  d["tile"] = c.tile;
  d["box_rows"] = c.box_rows;
  d["ctas"] = c.ctas;
  return d;
}

// ------------------------------------------------------------------ rows
int by_token(const at::Tensor& x, const Routing& r, const char* what) {
  const int type = matrix(x, what);
  if (x.size(0) != r.c.tokens || x.device() != r.device())
    value_error(std::string(what) + " must have a row for each of the routing's " +
                std::to_string(r.c.tokens) + " tokens, on its device");
  return type;
}

int by_slot(const at::Tensor& y, const Routing& r, const char* what) {
  const int type = matrix(y, what);
  if (y.size(0) != r.slots() || !y.is_contiguous() || y.device() != r.device())
    value_error(std::string(what) + " must be contiguous with a row for each of the routing's " +
                std::to_string(r.slots()) + " slots, on its device");
  return type;
}

const float* weights_of(const at::Tensor& w, const Routing& r) {
  if (w.scalar_type() != at::kFloat) type_error("weights must be float32");
  if (w.sizes() != r.ids.sizes() || !w.is_contiguous() || w.device() != r.device())
    value_error("weights must be contiguous, of the routing's tokens x top_k, on its device");
  return static_cast<const float*>(w.data_ptr());
}

at::Tensor dispatch(const at::Tensor& x, const Routing& r, const Out& out,
                    const py::object& stream) {
  const int type = by_token(x, r, "x");
  const On on(x.device(), stream);
  const at::Tensor y = output(out, r.slots(), x.size(1), x.scalar_type(), x.device());
  check(moe_dispatch(y.data_ptr(), x.data_ptr(), row_stride(x), x.size(1), type, &r.c, on.stream()),
        "moe_dispatch");
  return y;
}

at::Tensor dispatch_backward(const at::Tensor& grad_y, const Routing& r, const Out& out,
                             const py::object& stream) {
  const int type = by_slot(grad_y, r, "grad_y");
  const On on(grad_y.device(), stream);
  const at::Tensor x =
      output(out, r.c.tokens, grad_y.size(1), grad_y.scalar_type(), grad_y.device());
  check(moe_dispatch_backward(x.data_ptr(), grad_y.data_ptr(), grad_y.size(1), type, &r.c,
                              on.stream()),
        "moe_dispatch_backward");
  return x;
}

at::Tensor combine(const at::Tensor& y, const Routing& r, const at::Tensor& weights,
                   const Out& out, const py::object& stream) {
  const int type = by_slot(y, r, "y");
  const float* const w = weights_of(weights, r);
  const On on(y.device(), stream);
  const at::Tensor o = output(out, r.c.tokens, y.size(1), y.scalar_type(), y.device());
  check(moe_combine(o.data_ptr(), y.data_ptr(), w, y.size(1), type, &r.c, on.stream()),
        "moe_combine");
  return o;
}

std::pair<at::Tensor, at::Tensor> combine_backward(const at::Tensor& grad_out, const at::Tensor& y,
                                                   const Routing& r, const at::Tensor& weights,
                                                   const py::object& stream) {
  const int type = by_slot(y, r, "y");
  if (by_token(grad_out, r, "grad_out") != type || grad_out.size(1) != y.size(1) ||
      !grad_out.is_contiguous())
    value_error("grad_out must be contiguous, of y's type and width");
  const float* const w = weights_of(weights, r);
  const On on(y.device(), stream);
  const at::Tensor grad_y = fresh(y.sizes(), y.scalar_type(), y.device());
  const at::Tensor grad_w = fresh({r.c.tokens, r.c.top_k}, at::kFloat, y.device());
  check(moe_combine_backward(grad_y.data_ptr(), static_cast<float*>(grad_w.data_ptr()),
                             grad_out.data_ptr(), y.data_ptr(), w, y.size(1), type, &r.c,
                             on.stream()),
        "moe_combine_backward");
  return {grad_y, grad_w};
}

}  // namespace

#include "linear_binding.h"

PYBIND11_MODULE(_experts, m) {
  const auto none = py::none();
  py::class_<Routing, RoutingPtr>(m, "Routing",
                                  "Where each slot (token, j) went: rows[token, j] is its row in "
                                  "expert order, and expert e has rows "
                                  "offsets[e] to offsets[e + 1] - 1.  Dropped slots have the rows "
                                  "from offsets[-1] on.  All int32, on the device.  moe_sort makes "
                                  "one; a program with a router of its own can give the tensors "
                                  "itself (rows: a permutation of the slots; offsets: from 0, "
                                  "non-decreasing; neither is checked).  What ids holds "
                                  "after that does not matter: no call reads it again.")
      .def(py::init(&given_routing), py::arg("offsets"), py::arg("rows"), py::arg("ids"))
      .def_property_readonly("offsets", &Routing::get_offsets)
      .def_property_readonly("rows", &Routing::get_rows)
      .def_readonly("ids", &Routing::ids)
      .def_property_readonly("tokens", [](const Routing& r) { return r.c.tokens; })
      .def_property_readonly("top_k", [](const Routing& r) { return r.c.top_k; })
      .def_property_readonly("experts", [](const Routing& r) { return r.c.experts; })
      .def_property_readonly("slots", &Routing::slots);
  py::class_<Fp4Matrix, MatrixPtr>(
      m, "Fp4Matrix",
      "A matrix of 4-bit blocks in the layout of include/moe_fp4.h.\n\n"
      "codes: rows x (cols rounded up to 32) / 2 bytes.  scales: tiles x chunks x 512 bytes.\n"
      "group_rows: rows of each group (for weights of several experts, one expert's outputs;\n"
      "default: all rows are one group).  Instead, `routing` marks rows in expert order.")
      .def(py::init(&given_matrix), py::arg("codes"), py::arg("scales"), py::kw_only(),
           py::arg("cols"), py::arg("format") = "nvfp4", py::arg("exponent") = 0,
           py::arg("group_rows") = none, py::arg("routing") = none)
      .def_property_readonly("codes", &Fp4Matrix::get_codes)
      .def_property_readonly("scales", &Fp4Matrix::get_scales)
      .def_readonly("routing", &Fp4Matrix::routing)
      .def_property_readonly("rows", [](const Fp4Matrix& q) { return q.c.rows; })
      .def_property_readonly("cols", [](const Fp4Matrix& q) { return q.c.cols; })
      .def_property_readonly("format", [](const Fp4Matrix& q) { return format_name(q.c.format); })
      .def_property_readonly("exponent", [](const Fp4Matrix& q) { return q.c.exponent; })
      .def_property_readonly("groups", [](const Fp4Matrix& q) { return q.c.groups; })
      .def_property_readonly("group_rows", [](const Fp4Matrix& q) { return q.c.group_rows; });

  m.def("fp4_quantize", &quantize, py::arg("x"), py::kw_only(), py::arg("format") = "nvfp4",
        py::arg("exponent") = 0, py::arg("group_rows") = none, py::arg("routing") = none,
        py::arg("out") = none, py::arg("stream") = none,
        "x (rows x cols, float16 or bfloat16, rows contiguous) as an Fp4Matrix.\n\n"
        "With a routing, x has a row per token and the result a row per slot, in expert order.");
  m.def("fp4_dequantize", &dequantize, py::arg("q"), py::arg("dtype") = none,
        py::arg("out") = none, py::arg("stream") = none,
        "The values of q, rows x cols (float16 unless dtype says bfloat16); rows of dropped slots "
        "are zero.");
  m.def("fp4_gemm_tn", &gemm, py::arg("a"), py::arg("b"), py::kw_only(), py::arg("alpha") = 1.0,
        py::arg("dtype") = none, py::arg("out") = none, py::arg("stream") = none,
        py::arg("timeout_ns") = 0, py::arg("inject") = 0,
        "out[r] = alpha * a[r] @ b[g(r)]^T (fp32 accumulation; float16 unless dtype says bfloat16): "
        "g(r) is the group of row r, so with activations in expert order each row meets its "
        "expert's weights; rows of dropped slots give zeros.  b has as many groups as a, each of "
        "b.group_rows outputs.  timeout_ns and inject: see fp4_gemm_tn_ex in moe_fp4.h.");
  m.def("fp4_get_device_error",
        [](const py::object& stream) { return device_error(stream, fp4_get_device_error); },
        py::arg("stream") = none,
        "(status, raw word) of the stream's error word of fp4_gemm_tn; synchronises the stream.");
  m.def("fp4_scale_bytes", &scale_bytes, py::arg("rows"), py::arg("cols"),
        py::arg("format") = "nvfp4", py::arg("groups") = 1, py::arg("by_offsets") = false,
        "Bytes of an Fp4Matrix's scales.");
  m.def("fp4_query_config", &query_config, py::arg("rows"), py::arg("n"), py::arg("cols"),
        py::arg("format") = "nvfp4", py::arg("groups") = 1, py::arg("by_offsets") = false,
        "The form that fp4_gemm_tn takes for a product of these sizes, without running it.");
  m.def("moe_sort", &sort, py::arg("ids"), py::arg("experts"), py::arg("stream") = none,
        "Slots sorted by expert.  ids: tokens x top_k int32; a number outside [0, experts) drops "
        "its slot.  The order within an expert is the slots' own.");
  m.def("moe_pairs", &pairs_of, py::arg("routing"), py::arg("stream") = none,
        "The slot (token * top_k + j) of each row: the inverse of the routing's rows.");
  m.def("moe_dispatch", &dispatch, py::arg("x"), py::arg("routing"), py::arg("out") = none,
        py::arg("stream") = none,
        "x's rows (a row per token) in expert order, a row per slot; zeros for dropped slots.");
  m.def("moe_dispatch_backward", &dispatch_backward, py::arg("grad_y"), py::arg("routing"),
        py::arg("out") = none, py::arg("stream") = none,
        "moe_dispatch's gradient: each token's sum over its kept slots.");
  m.def("moe_combine", &combine, py::arg("y"), py::arg("routing"), py::arg("weights"),
        py::arg("out") = none, py::arg("stream") = none,
        "Each token's weighted sum of its kept slots' rows of y.  weights: tokens x top_k float32.");
  m.def("moe_combine_backward", &combine_backward, py::arg("grad_out"), py::arg("y"),
        py::arg("routing"), py::arg("weights"), py::arg("stream") = none,
        "moe_combine's gradients: (of y, of weights); zeros for dropped slots.");

  define_linear(m);
}
