// Python binding of the residual-stream operators: the argument checks, output
// allocation and C calls of sandwich_rms, embedding_lookup and their gradients,
// against PyTorch's C++ interface.  It computes nothing.
//
// These calls are made for single rows as well, where the call is all host
// time: through ctypes a one-row sandwich_rms cost 24 us of it, of which the
// library's own part is 2.
//
// Messages and exception types follow the ctypes wrappers in ops.py: ValueError
// for shapes, strides and devices, TypeError for dtypes, NormError for what the
// library refuses.

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <optional>
#include <string>

#include "norm.h"

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

namespace {

[[noreturn]] void value_error(const std::string& m) { throw py::value_error(m); }
[[noreturn]] void type_error(const std::string& m) { throw py::type_error(m); }

std::string name_of(at::ScalarType t) { return c10::toString(t); }

bool dtype_code(at::ScalarType t, norm_dtype* out) {
  switch (t) {
    case at::kFloat: *out = NORM_F32; return true;
    case at::kBFloat16: *out = NORM_BF16; return true;
    case at::kHalf: *out = NORM_F16; return true;
    default: return false;
  }
}

norm_dtype code(at::ScalarType t, const char* what) {
  norm_dtype c;
  if (!dtype_code(t, &c))
    type_error(std::string(what) + ": dtype " + name_of(t) + " not supported (float32, bfloat16 or float16)");
  return c;
}

const Tensor& cuda_tensor(const Tensor& t, const char* what) {
  if (!t.defined() || !t.is_cuda()) value_error(std::string(what) + " must be a CUDA tensor");
  return t;
}

// A row tensor: N rows of H contiguous elements, ld apart.
struct Rows {
  void* p = nullptr;
  int64_t N = 0, H = 0, ld = 0;
};

// The rows of a tensor on any device.
Rows row_view(const Tensor& t, const char* what) {
  const int64_t d = t.dim();
  if (d < 1) value_error(std::string(what) + " must have at least one dim");
  Rows r;
  r.p = t.data_ptr();
  r.H = t.size(d - 1);
  if (r.H > 1 && t.stride(d - 1) != 1) value_error(std::string(what) + ": the last dim must be contiguous");
  r.N = 1;
  // The innermost dim of several rows gives the row stride; every dim outside
  // it has to start where the ones inside end (`reach`).  An expanded dim has
  // stride 0 and counts like any other: beside a dim with another stride it does
  // not flatten, and a row stride of 0 is refused by the library.
  bool seen = false, flat = true;
  int64_t ld = 0, reach = 0;
  for (int64_t i = d - 2; i >= 0; --i) {
    const int64_t n = t.size(i);
    r.N *= n;
    if (n <= 1) continue;
    if (!seen) {
      seen = true;
      ld = reach = t.stride(i);
    } else if (t.stride(i) != reach) {
      flat = false;
    }
    reach *= n;
  }
  if (r.N > 1 && !flat) value_error(std::string(what) + ": leading dims do not flatten to one row stride");
  r.ld = r.N > 1 ? ld : std::max<int64_t>(r.H, 1);
  return r;
}

Rows rows(const Tensor& t, const char* what) { return row_view(cuda_tensor(t, what), what); }

// A tensor that matches the rows of `ref`.
Rows like(const Tensor& t, const Tensor& ref, const Rows& of, const char* what) {
  const Rows r = rows(t, what);
  if (r.N != of.N || r.H != of.H || t.scalar_type() != ref.scalar_type() || t.device() != ref.device())
    value_error(std::string(what) + " must match the rows, width, dtype (" + name_of(ref.scalar_type()) + ") and device (" +
                ref.device().str() + ") of the input");
  return r;
}

const void* vec(const Opt& t, int64_t H, const char* what, const Tensor& ref) {
  if (!t) return nullptr;
  if (!t->is_cuda() || t->dim() != 1 || t->size(0) != H || (H > 1 && t->stride(0) != 1))
    value_error(std::string(what) + " must be a contiguous CUDA tensor of shape (" + std::to_string(H) + ",)");
  if (t->device() != ref.device())
    value_error(std::string(what) + " is on " + t->device().str() + ", the rows on " + ref.device().str());
  code(t->scalar_type(), what);
  return t->data_ptr();
}

const float* stats(const Opt& t, int64_t N, const char* what, const Tensor& ref) {
  if (!t) return nullptr;
  cuda_tensor(*t, what);
  if (t->scalar_type() != at::kFloat) value_error(std::string(what) + " must be float32, not " + name_of(t->scalar_type()));
  if (t->numel() != N || !t->is_contiguous())
    value_error(std::string(what) + " must be a contiguous tensor of " + std::to_string(N) + " elements (one per row)");
  if (t->device() != ref.device())
    value_error(std::string(what) + " is on " + t->device().str() + ", the rows on " + ref.device().str());
  return t->data_ptr<float>();
}

// The dtype two parameters share, or `other` where both are absent.
at::ScalarType shared_dtype(const Opt& a, const Opt& b, at::ScalarType other) {
  if (a && b && a->scalar_type() != b->scalar_type()) type_error("gamma_post and gamma_pre must share a dtype");
  return a ? a->scalar_type() : b ? b->scalar_type() : other;
}

struct Gate {
  const void* p = nullptr;
  int64_t rows = 0, ld = 0;
  norm_dtype dt = NORM_F32;
};

// Whether `t` would broadcast over an outer dim of `ref` and follow a dim inside
// it, as (1, T, H) does against (B, T, H).  Gate rows serve runs of consecutive
// rows, which is something else.
bool broadcasts_outer(const Tensor& t, const Tensor& ref) {
  if (t.dim() != ref.dim()) return false;
  bool open = false, follows = false;
  for (int64_t i = 0; i + 1 < t.dim(); ++i) {
    if (t.size(i) != ref.size(i) && t.size(i) != 1) return false;
    if (t.size(i) == ref.size(i))
      follows |= open && ref.size(i) > 1;
    else
      open = true;
  }
  return follows;
}

Gate gate_view(const Opt& t, const Rows& of, const Tensor& ref) {
  Gate g;
  g.dt = code(ref.scalar_type(), "x");
  if (!t) return g;
  const Rows r = rows(*t, "gate");
  if (r.H != of.H || t->device() != ref.device())
    value_error("gate must have " + std::to_string(of.H) + " columns on " + ref.device().str());
  if (broadcasts_outer(*t, ref))
    value_error("gate: a row serves a run of consecutive rows; dims that follow a broadcast one are not taken");
  const bool none = r.N == 0 && of.N == 0;  // no sequences: no gate rows, and nothing reads one
  if (!none && (r.N < 1 || of.N % r.N != 0 || (of.N > 0 && r.N > of.N)))
    value_error("gate has " + std::to_string(r.N) + " rows, which do not divide the " + std::to_string(of.N) +
                " rows into equal runs");
  const norm_dtype c = code(t->scalar_type(), "gate");
  if (c != g.dt && c != NORM_F32)
    type_error("gate: dtype " + name_of(t->scalar_type()) + " must be the rows' or float32");
  if (none) return g;
  g.p = r.p;
  g.rows = r.N;
  g.ld = r.ld;
  g.dt = c;
  return g;
}

Tensor new_like(const Tensor& x) { return at::empty(x.sizes(), x.options().requires_grad(false)); }
Tensor new_vec(int64_t n, const Tensor& ref, at::ScalarType t) { return at::empty({n}, ref.options().dtype(t).requires_grad(false)); }

py::object obj(const Tensor& t) { return t.defined() ? py::cast(t) : py::object(py::none()); }

norm_stream_t stream_of(const Tensor& t) {
  return reinterpret_cast<norm_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

void check(const char* fn, norm_status st) {
  if (st != NORM_OK) py::module_::import("rmsnorm_ln_fwd_gb300._lib").attr("check")(fn, (int)st);
}

// A caller's workspace, or a fresh one of `need` bytes.
Tensor workspace_of(const Opt& ws, size_t need, const Tensor& ref, size_t* bytes) {
  if (need == 0) throw std::runtime_error("could not size the workspace (no CUDA device?)");
  if (!ws) {
    *bytes = need;
    return at::empty({(int64_t)need}, ref.options().dtype(at::kByte).requires_grad(false));
  }
  if (!ws->is_cuda() || ws->device() != ref.device() || !ws->is_contiguous())
    value_error("workspace must be a contiguous CUDA tensor on " + ref.device().str());
  *bytes = (size_t)ws->numel() * (size_t)ws->element_size();
  return *ws;
}

py::tuple sandwich_rms_(const Tensor& x, const Tensor& residual, const Opt& gamma_post, const Opt& gate,
                        const Opt& gamma_pre, double eps, double residual_scale, bool post, bool pre, const Opt& h_out,
                        const Opt& out, bool save_stats) {
  const Rows xr = rows(x, "x");
  const norm_dtype xc = code(x.scalar_type(), "x");
  const Rows rr = like(residual, x, xr, "residual");
  if ((gamma_post && !post) || (!pre && (gamma_pre || out)))
    value_error("gamma_post needs post_norm; gamma_pre and out need pre_norm");
  const void* gpost = vec(gamma_post, xr.H, "gamma_post", x);
  const void* gpre = vec(gamma_pre, xr.H, "gamma_pre", x);
  const norm_dtype wc = code(shared_dtype(gamma_post, gamma_pre, x.scalar_type()), "gamma");
  const Gate g = gate_view(gate, xr, x);
  const c10::cuda::CUDAGuard guard(x.device());
  const Tensor h = h_out ? *h_out : new_like(x);
  const Rows hr = h_out ? like(h, x, xr, "h_out") : Rows{h.data_ptr(), xr.N, xr.H, std::max<int64_t>(xr.H, 1)};
  Tensor y, rpost, rpre;
  Rows yr;
  if (pre) {
    y = out ? *out : new_like(x);
    yr = out ? like(y, x, xr, "out") : Rows{y.data_ptr(), xr.N, xr.H, std::max<int64_t>(xr.H, 1)};
  }
  if (save_stats && post) rpost = new_vec(xr.N, x, at::kFloat);
  if (save_stats && pre) rpre = new_vec(xr.N, x, at::kFloat);
  const unsigned norms = (post ? NORM_SANDWICH_POST : 0u) | (pre ? NORM_SANDWICH_PRE : 0u);
  check("sandwich_rms",
        sandwich_rms(xr.p, xr.ld, rr.p, rr.ld, gpost, g.p, g.ld, g.rows, gpre, yr.p, yr.ld, hr.p, hr.ld,
                     rpost.defined() ? rpost.data_ptr<float>() : nullptr, rpre.defined() ? rpre.data_ptr<float>() : nullptr,
                     xr.N, xr.H, (float)eps, (float)residual_scale, norms, xc, wc, g.dt, stream_of(x)));
  return py::make_tuple(obj(y), obj(h), obj(rpost), obj(rpre));
}

py::tuple sandwich_rms_grad_(const Opt& dy, const Tensor& x, const Opt& h, const Opt& rstd_post, const Opt& rstd_pre,
                             const Opt& gamma_post, const Opt& gate, const Opt& gamma_pre, const Opt& dh_in,
                             double residual_scale, bool need_param_grads, const Opt& workspace, const Opt& dx,
                             const Opt& dres, std::optional<at::ScalarType> param_dtype) {
  const Rows xr = rows(x, "x");
  const norm_dtype xc = code(x.scalar_type(), "x");
  const bool post = rstd_post.has_value(), pre = rstd_pre.has_value();
  if (pre != dy.has_value() || pre != h.has_value())
    value_error("dy, h and rstd_pre come together (all None without the norm after the add)");
  if ((!post && gamma_post) || (!pre && gamma_pre)) value_error("gamma_post needs rstd_post; gamma_pre needs rstd_pre");
  if (!post && !pre) value_error("rstd_post and rstd_pre are both None: no norm to differentiate");
  if (!dy && !dh_in) value_error("dy and dh_in are both None: no gradient arrives");
  const Rows dyr = pre ? like(*dy, x, xr, "dy") : Rows();
  const Rows hr = pre ? like(*h, x, xr, "h") : Rows();
  const Rows dir = dh_in ? like(*dh_in, x, xr, "dh_in") : Rows();
  const float* rpost = stats(rstd_post, xr.N, "rstd_post", x);
  const float* rpre = stats(rstd_pre, xr.N, "rstd_pre", x);
  const void* gpost = vec(gamma_post, xr.H, "gamma_post", x);
  const void* gpre = vec(gamma_pre, xr.H, "gamma_pre", x);
  const at::ScalarType wt = shared_dtype(gamma_post, gamma_pre, param_dtype.value_or(x.scalar_type()));
  const norm_dtype wc = code(wt, "param_dtype");
  const Gate g = gate_view(gate, xr, x);
  const c10::cuda::CUDAGuard guard(x.device());
  const Tensor odx = dx ? *dx : new_like(x);
  const Rows dxr = dx ? like(odx, x, xr, "dx") : Rows{odx.data_ptr(), xr.N, xr.H, std::max<int64_t>(xr.H, 1)};
  const Tensor odr = dres ? *dres : new_like(x);
  const Rows drr = dres ? like(odr, x, xr, "dres") : Rows{odr.data_ptr(), xr.N, xr.H, std::max<int64_t>(xr.H, 1)};
  Tensor dgpost, dgate, dgpre, ws;
  size_t wsb = 0;
  if (need_param_grads) {
    if (post) dgpost = new_vec(xr.H, x, wt);
    if (pre) dgpre = new_vec(xr.H, x, wt);
    if (gate) dgate = new_like(*gate);
    ws = workspace_of(workspace, sandwich_rms_workspace_bytes(xr.H, g.rows, x.get_device()), x, &wsb);
  }
  const unsigned norms = (post ? NORM_SANDWICH_POST : 0u) | (pre ? NORM_SANDWICH_PRE : 0u);
  auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  check("sandwich_rms_grad",
        sandwich_rms_grad(dyr.p, dyr.ld, xr.p, xr.ld, hr.p, hr.ld, rpost, rpre, gpost, g.p, g.ld, g.rows, gpre, dir.p,
                          dir.ld, dxr.p, dxr.ld, drr.p, drr.ld, ptr(dgpost), ptr(dgate), xr.H, ptr(dgpre), ptr(ws), wsb,
                          xr.N, xr.H, (float)residual_scale, norms, xc, wc, g.dt, stream_of(x)));
  return py::make_tuple(obj(odx), obj(odr), obj(dgpost), obj(dgate), obj(dgpre));
}

norm_itype tokens_of(const Tensor& tokens, const Tensor& ref) {
  cuda_tensor(tokens, "tokens");
  const at::ScalarType t = tokens.scalar_type();
  if (t != at::kInt && t != at::kLong) type_error("tokens: dtype " + name_of(t) + " not supported (int32 or int64)");
  if (!tokens.is_contiguous()) value_error("tokens must be contiguous");
  if (tokens.device() != ref.device())
    value_error("tokens are on " + tokens.device().str() + ", the rows on " + ref.device().str());
  return t == at::kLong ? NORM_I64 : NORM_I32;
}

Rows table_of(const Tensor& t, const char* what) {
  cuda_tensor(t, what);
  if (t.dim() != 2) value_error(std::string(what) + " must have two dims (rows, columns)");
  return rows(t, what);
}

// One row a token: the caller's tensor, or a fresh one of tokens' shape.
Tensor token_rows(const Opt& out, const Tensor& tokens, const Tensor& table, int64_t H, const char* what, Rows* r) {
  if (!out) {
    std::vector<int64_t> shape(tokens.sizes().begin(), tokens.sizes().end());
    shape.push_back(H);
    const Tensor t = at::empty(shape, table.options().requires_grad(false));
    *r = Rows{t.data_ptr(), tokens.numel(), H, std::max<int64_t>(H, 1)};
    return t;
  }
  *r = rows(*out, what);
  if (r->N != tokens.numel() || r->H != H || out->scalar_type() != table.scalar_type() || out->device() != table.device())
    value_error(std::string(what) + " must have " + std::to_string(tokens.numel()) + " rows of " + std::to_string(H) + " " +
                name_of(table.scalar_type()) + " columns on " + table.device().str());
  return *out;
}

py::object embedding_lookup_(const Tensor& tokens, const Tensor& table, double scale, const Opt& out) {
  const Rows tr = table_of(table, "table");
  const norm_dtype xc = code(table.scalar_type(), "table");
  const norm_itype it = tokens_of(tokens, table);
  const c10::cuda::CUDAGuard guard(table.device());
  Rows hr;
  const Tensor h = token_rows(out, tokens, table, tr.H, "out", &hr);
  check("embedding_lookup", embedding_lookup(tr.p, tr.ld, tr.N, tokens.data_ptr(), it, hr.p, hr.ld, hr.N, tr.H, (float)scale,
                                             xc, stream_of(table)));
  return obj(h);
}

py::tuple embedding_rms_(const Tensor& tokens, const Tensor& table, const Opt& gamma, double eps, double scale,
                         const Opt& h_out, const Opt& out, bool save_stats) {
  const Rows tr = table_of(table, "table");
  const norm_dtype xc = code(table.scalar_type(), "table");
  const norm_itype it = tokens_of(tokens, table);
  const void* g = vec(gamma, tr.H, "gamma", table);
  const norm_dtype wc = gamma ? code(gamma->scalar_type(), "gamma") : xc;
  const c10::cuda::CUDAGuard guard(table.device());
  Rows hr, yr;
  const Tensor h = token_rows(h_out, tokens, table, tr.H, "h_out", &hr);
  const Tensor y = token_rows(out, tokens, table, tr.H, "out", &yr);
  const Tensor rstd = save_stats ? new_vec(hr.N, table, at::kFloat) : Tensor();
  check("embedding_rms",
        embedding_rms(tr.p, tr.ld, tr.N, tokens.data_ptr(), it, g, yr.p, yr.ld, hr.p, hr.ld,
                      save_stats ? rstd.data_ptr<float>() : nullptr, hr.N, tr.H, (float)eps, (float)scale, xc, wc,
                      stream_of(table)));
  return py::make_tuple(obj(y), obj(h), obj(rstd));
}

py::object embedding_grad_(const Tensor& dh, const Tensor& tokens, int64_t num_rows, double scale,
                           std::optional<int64_t> padding_idx, const Opt& out, bool accumulate,
                           std::optional<at::ScalarType> param_dtype, const Opt& workspace) {
  const Rows dr = rows(dh, "dh");
  const norm_dtype xc = code(dh.scalar_type(), "dh");
  const norm_itype it = tokens_of(tokens, dh);
  if (tokens.numel() != dr.N)
    value_error("dh has " + std::to_string(dr.N) + " rows for " + std::to_string(tokens.numel()) + " tokens");
  if (padding_idx && (*padding_idx < 0 || *padding_idx >= num_rows))
    value_error("padding_idx " + std::to_string(*padding_idx) + " is not a row of the table");
  if (!out && accumulate) value_error("accumulate needs out");
  if (num_rows < 0) value_error("num_rows must not be negative");
  const c10::cuda::CUDAGuard guard(dh.device());
  const Tensor table =
      out ? *out : at::empty({num_rows, dr.H}, dh.options().dtype(param_dtype.value_or(dh.scalar_type())).requires_grad(false));
  const Rows tr = table_of(table, "out");
  if (tr.N != num_rows || tr.H != dr.H || table.device() != dh.device())
    value_error("out must be (" + std::to_string(num_rows) + ", " + std::to_string(dr.H) + ") on " + dh.device().str());
  const norm_dtype wc = code(table.scalar_type(), "out");
  size_t wsb = 0;
  const Tensor ws = workspace_of(workspace, embedding_grad_workspace_bytes(dr.N, dr.H), dh, &wsb);
  check("embedding_grad", embedding_grad(dr.p, dr.ld, tokens.data_ptr(), it, tr.p, tr.ld, tr.N, ws.data_ptr(), wsb, dr.N, dr.H,
                                         (float)scale, padding_idx.value_or(-1), accumulate, xc, wc, stream_of(dh)));
  return obj(table);
}

}  // namespace

// The PyTorch this is compiled against, found in the file before it is loaded.
extern "C" __attribute__((used)) const char norm_bind_torch[];
const char norm_bind_torch[] = "norm_bind_torch=" NORM_BIND_TORCH;

PYBIND11_MODULE(_bind, m) {
  m.def("row_view", [](const Tensor& t) {  // (N, H, ld) of a tensor on any device, for tests
    const Rows r = row_view(t, "t");
    return py::make_tuple(r.N, r.H, r.ld);
  });
  m.def("sandwich_rms", &sandwich_rms_);
  m.def("sandwich_rms_grad", &sandwich_rms_grad_);
  m.def("embedding_lookup", &embedding_lookup_);
  m.def("embedding_rms", &embedding_rms_);
  m.def("embedding_grad", &embedding_grad_);
}
