// The binding of linear.h, part of experts_binding.cpp (which has the checks and
// the routing that both use).
#include "linear.h"

namespace {

using Form = std::optional<std::tuple<int, int, int>>;  // cta_pair, tile, split_k

int activation_of(const std::string& name) {
  const char* const names[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};
  for (int i = 0; i < 5; ++i)
    if (name == names[i]) return i;
  value_error("unknown activation '" + name + "'");
}

linear_options_t options_of(const Form& form, uint64_t timeout_ns, int inject) {
  linear_options_t o{};
  if (form) std::tie(o.cta_pair, o.tile, o.split_k) = *form;
  o.inject = inject;
  o.timeout_ns = timeout_ns;
  return o;
}

[[noreturn]] void does_not_fit(const char* what, const std::string& wanted) {
  value_error(std::string(what) + " must be " + wanted + ", of x's type and on its device");
}

// The layer's weights: out x in, or experts x out x in with a routing.
struct Layer {
  linear_t c{};
  at::ScalarType type = at::kHalf;
  at::Device device{at::kCUDA};

  void of_rows(const at::Tensor& t, const char* what) {  // x, or the output's gradient
    c.type = matrix(t, what);
    c.rows = t.size(0);
    type = t.scalar_type();
    device = t.device();
  }

  void with_routing(const Routing* r, const char* what) {
    if (!r) return;
    if (c.rows != r->slots() || device != r->device())
      value_error(std::string(what) + " must have a row for each of the routing's " +
                  std::to_string(r->slots()) + " slots, on its device");
    c.routing = &r->c;
  }

  void with_weight(const at::Tensor& w) {
    if (type_of(w.scalar_type(), "weight") != c.type || w.device() != device)
      value_error("weight must be of x's type and on its device");
    if (!c.routing) {
      matrix(w, "weight");
      c.out = w.size(0);
      c.in = w.size(1);
      c.ldw = row_stride(w);
    } else {
      if (w.dim() != 3 || w.size(0) != c.routing->experts)
        value_error("weight must be " + std::to_string(c.routing->experts) +
                    " x out x in, an expert's after the other's");
      c.out = w.size(1);
      c.in = w.size(2);
      c.ldw = w.size(1) > 1 ? w.stride(1) : w.size(0) > 1 ? w.stride(0) : c.in;
      if (w.numel() && ((c.in > 1 && w.stride(2) != 1) || c.ldw < c.in ||
                        (w.size(0) > 1 && w.stride(0) != c.out * c.ldw)))
        value_error("weight's rows must be contiguous, an expert's after the other's");
    }
    c.w = w.data_ptr();
  }

  void with_x(const at::Tensor& x) {
    c.x = x.data_ptr();
    c.ldx = row_stride(x);
  }

  int64_t experts() const { return c.routing ? c.routing->experts : 1; }

  // The bias (or its gradient): `out` elements, with a routing for each expert.
  const void* bias_of(const Out& b) const {
    if (!b) return nullptr;
    const bool fits = c.routing ? b->dim() == 2 && b->size(0) == experts() && b->size(1) == c.out
                                : b->dim() == 1 && b->size(0) == c.out;
    if (!fits || b->scalar_type() != type || !b->is_contiguous() || b->device() != device)
      does_not_fit("bias", c.routing ? "contiguous, experts x out" : "contiguous, `out` elements");
    return b->data_ptr();
  }

  // A matrix of rows x out besides, whose rows may be apart.
  int64_t beside(const at::Tensor& t, const char* what) const {
    if (matrix(t, what) != c.type || t.size(0) != c.rows || t.size(1) != c.out ||
        t.device() != device)
      does_not_fit(what, std::to_string(c.rows) + " x " + std::to_string(c.out));
    return row_stride(t);
  }

  at::Tensor workspace(uint64_t bytes) const {
    return bytes ? fresh({static_cast<int64_t>(bytes)}, at::kByte, device) : at::Tensor();
  }
};

py::object forward(const at::Tensor& x, const Routing* routing, const at::Tensor& weight,
                   const Out& bias, const std::string& activation, const Out& residual,
                   bool save_preact, const Out& out, const py::object& stream, const Form& form,
                   uint64_t timeout_ns, int inject) {
  Layer l;
  l.of_rows(x, "x");
  l.c.activation = activation_of(activation);
  l.with_routing(routing, "x");
  l.with_weight(weight);
  if (x.size(1) != l.c.in)
    value_error("x has rows of " + std::to_string(x.size(1)) + ", the weights of " +
                std::to_string(l.c.in));
  l.with_x(x);
  const void* const b = l.bias_of(bias);
  const int64_t ldr = residual ? l.beside(*residual, "residual") : 0;
  const On on(l.device, stream);
  const at::Tensor o = output(out, l.c.rows, l.c.out, l.type, l.device);
  const at::Tensor z = save_preact ? fresh({l.c.rows, l.c.out}, l.type, l.device) : at::Tensor();
  const linear_options_t opt = options_of(form, timeout_ns, inject);
  uint64_t bytes = 0;
  check(linear_forward_workspace(&l.c, &opt, &bytes), "linear");
  const at::Tensor space = l.workspace(bytes);
  check(linear_forward(o.data_ptr(), save_preact ? z.data_ptr() : nullptr, &l.c, b,
                       residual ? residual->data_ptr() : nullptr, ldr,
                       bytes ? space.data_ptr() : nullptr, bytes, &opt, on.stream()),
        "linear");
  if (save_preact) return py::make_tuple(o, z);
  return py::cast(o);
}

py::tuple backward(const at::Tensor& grad_out, const Out& x, const Routing* routing,
                   const Out& weight, const Out& preact, const std::string& activation,
                   bool need_x, bool need_weight, bool need_bias, const py::object& stream,
                   const Form& form, uint64_t timeout_ns, int inject) {
  Layer l;
  l.of_rows(grad_out, "grad_out");
  l.c.activation = activation_of(activation);
  l.with_routing(routing, "grad_out");
  l.c.out = grad_out.size(1);
  if (need_x && !weight) value_error("the gradient of x needs the weights");
  if (need_weight && !x) value_error("the gradient of the weights needs x");
  if (weight) {
    l.with_weight(*weight);
    if (l.c.out != grad_out.size(1))
      value_error("grad_out has rows of " + std::to_string(grad_out.size(1)) +
                  ", the weights give " + std::to_string(l.c.out));
  }
  if (x) {
    if (matrix(*x, "x") != l.c.type || x->size(0) != l.c.rows || x->device() != l.device ||
        (weight && x->size(1) != l.c.in))
      value_error("x must have a row for each of grad_out's, as long as the weights', of its type "
                  "and on its device");
    l.c.in = x->size(1);
    l.with_x(*x);
  }
  const void* z = nullptr;
  if (l.c.activation != LINEAR_NONE) {
    if (!preact) value_error("the gradient of " + activation + " needs preact");
    l.beside(*preact, "preact");
    if (!preact->is_contiguous()) value_error("preact must be contiguous");
    z = preact->data_ptr();
  }
  const On on(l.device, stream);
  Out grad_x, grad_w, grad_b;
  if (need_x) grad_x = fresh({l.c.rows, l.c.in}, l.type, l.device);
  if (need_weight)
    grad_w = l.c.routing ? fresh({l.experts(), l.c.out, l.c.in}, l.type, l.device)
                         : fresh({l.c.out, l.c.in}, l.type, l.device);
  if (need_bias)
    grad_b = l.c.routing ? fresh({l.experts(), l.c.out}, l.type, l.device)
                         : fresh({l.c.out}, l.type, l.device);
  const auto at = [](const Out& t) { return t ? t->data_ptr() : nullptr; };
  const int64_t ldg = row_stride(grad_out);
  uint64_t bytes = 0;
  check(linear_backward_workspace(at(grad_x), at(grad_w), at(grad_b), &l.c, grad_out.data_ptr(),
                                  ldg, &bytes),
        "linear_backward");
  const at::Tensor space = l.workspace(bytes);
  const linear_options_t opt = options_of(form, timeout_ns, inject);
  check(linear_backward(at(grad_x), at(grad_w), at(grad_b), &l.c, grad_out.data_ptr(), ldg, z,
                        bytes ? space.data_ptr() : nullptr, bytes, &opt, on.stream()),
        "linear_backward");
  return py::make_tuple(grad_x, grad_w, grad_b);
}

py::dict linear_config(const std::string& product, int64_t rows, int64_t in, int64_t out,
                       int experts, bool both) {
  const int kind = product == "forward"  ? LINEAR_FORWARD
                   : product == "grad_x" ? (both ? LINEAR_GRAD_X_OF_BOTH : LINEAR_GRAD_X)
                   : product == "grad_w" ? (both ? LINEAR_GRAD_W_OF_BOTH : LINEAR_GRAD_W)
                                         : -1;
  linear_config_t c{};
  check(linear_query_config(kind, rows, in, out, experts, &c), "linear_query_config");
  py::dict d;
  d["cta_pair"] = c.cta_pair;
  d["tile"] = c.tile;
  d["split_k"] = c.split_k;
  d["ctas"] = c.ctas;
  return d;
}

void define_linear(py::module_& m) {
  const auto none = py::none();
  m.def(
      "linear",
      [](const at::Tensor& x, const at::Tensor& weight, const Out& bias,
         const std::string& activation, const Out& residual, bool save_preact, const Out& out,
         const py::object& stream, const Form& form, uint64_t timeout_ns, int inject) {
        return forward(x, nullptr, weight, bias, activation, residual, save_preact, out, stream,
                       form, timeout_ns, inject);
      },
      py::arg("x"), py::arg("weight"), py::arg("bias") = none, py::kw_only(),
      py::arg("activation") = "none", py::arg("residual") = none, py::arg("save_preact") = false,
      py::arg("out") = none, py::arg("stream") = none, py::arg("form") = none,
      py::arg("timeout_ns") = 0, py::arg("inject") = 0,
      "act(x @ weight^T + bias) + residual: x rows x in, weight out x in, bias `out` elements, "
      "residual rows x out, all float16 or all bfloat16; fp32 sums, rounded once.  activation: "
      "none, relu, gelu, gelu_tanh or silu.  With save_preact also the sums before the activation, "
      "as linear_backward takes them: (out, preact).  Records no gradients: linear_backward gives "
      "them.  form, timeout_ns and inject: linear_options_t of linear.h.");
  m.def(
      "moe_linear",
      [](const at::Tensor& x, const Routing& routing, const at::Tensor& weight, const Out& bias,
         const std::string& activation, bool save_preact, const Out& out, const py::object& stream,
         const Form& form, uint64_t timeout_ns, int inject) {
        return forward(x, &routing, weight, bias, activation, std::nullopt, save_preact, out,
                       stream, form, timeout_ns, inject);
      },
      py::arg("x"), py::arg("routing"), py::arg("weight"), py::arg("bias") = none, py::kw_only(),
      py::arg("activation") = "none", py::arg("save_preact") = false, py::arg("out") = none,
      py::arg("stream") = none, py::arg("form") = none, py::arg("timeout_ns") = 0,
      py::arg("inject") = 0,
      "linear with each row's expert's weights: x slots x in, in expert order (as moe_dispatch "
      "leaves it), weight experts x out x in, bias experts x out.  Rows of dropped slots give "
      "zeros.  Records no gradients: moe_linear_backward gives them.");
  m.def(
      "linear_backward",
      [](const at::Tensor& grad_out, const Out& x, const Out& weight, const Out& preact,
         const std::string& activation, bool need_x, bool need_weight, bool need_bias,
         const py::object& stream, const Form& form, uint64_t timeout_ns, int inject) {
        return backward(grad_out, x, nullptr, weight, preact, activation, need_x, need_weight,
                        need_bias, stream, form, timeout_ns, inject);
      },
      py::arg("grad_out"), py::arg("x"), py::arg("weight"), py::kw_only(), py::arg("preact") = none,
      py::arg("activation") = "none", py::arg("need_x") = true, py::arg("need_weight") = true,
      py::arg("need_bias") = false, py::arg("stream") = none, py::arg("form") = none,
      py::arg("timeout_ns") = 0, py::arg("inject") = 0,
      "linear's gradients (of x, weight, bias), None for those not needed; the residual's is "
      "grad_out.  preact: what linear kept, needed but for activation none.  x may be None "
      "without need_weight, weight without need_x.  grad_out act'(preact) is rounded to the "
      "type for the products.");
  m.def(
      "moe_linear_backward",
      [](const at::Tensor& grad_out, const Out& x, const Routing& routing, const Out& weight,
         const Out& preact, const std::string& activation, bool need_x, bool need_weight,
         bool need_bias, const py::object& stream, const Form& form, uint64_t timeout_ns,
         int inject) {
        return backward(grad_out, x, &routing, weight, preact, activation, need_x, need_weight,
                        need_bias, stream, form, timeout_ns, inject);
      },
      py::arg("grad_out"), py::arg("x"), py::arg("routing"), py::arg("weight"), py::kw_only(),
      py::arg("preact") = none, py::arg("activation") = "none", py::arg("need_x") = true,
      py::arg("need_weight") = true, py::arg("need_bias") = false, py::arg("stream") = none,
      py::arg("form") = none, py::arg("timeout_ns") = 0, py::arg("inject") = 0,
      "moe_linear's gradients (of x, weight, bias): an expert's are the sums over its own rows, "
      "zero for one without; rows of dropped slots have zeros in grad_x and count in nothing.");
  m.def("linear_query_config", &linear_config, py::arg("product"), py::arg("rows"),
        py::arg("in_features"), py::arg("out_features"), py::arg("experts") = 0,
        py::kw_only(), py::arg("both") = false,
        "The form that a product (forward, grad_x or grad_w) of a layer of these sizes takes, "
        "without running it; experts: 0 for a dense one; both: grad_x or grad_w in a call for "
        "both of them, where it may be another.");
  m.def(
      "linear_get_device_error",
      [](const py::object& stream) { return device_error(stream, linear_get_device_error); },
      py::arg("stream") = none,
      "(status, raw word) of the stream's error word of these calls; synchronises the stream.");
}

}  // namespace
