// Python binding of the residual-stream operators, of the per-head norm and of
// the log probabilities: the argument checks, output allocation and C calls of
// sandwich_rms, embedding_lookup, head_rms_rotary, token_logprobs and their
// gradients, against PyTorch's C++ interface.  It computes nothing.
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

// The rows of a tensor on any device; returns whether one row stride reaches them all.
bool row_layout(const Tensor& t, const char* what, Rows* out) {
  const int64_t d = t.dim();
  if (d < 1) value_error(std::string(what) + " must have at least one dim");
  Rows& r = *out;
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
  r.ld = r.N > 1 ? ld : std::max<int64_t>(r.H, 1);
  return r.N <= 1 || flat;
}

Rows row_view(const Tensor& t, const char* what) {
  Rows r;
  if (!row_layout(t, what, &r)) value_error(std::string(what) + ": leading dims do not flatten to one row stride");
  return r;
}

Rows rows(const Tensor& t, const char* what) { return row_view(cuda_tensor(t, what), what); }

void same_rows(const Tensor& t, const Rows& r, const Tensor& ref, const Rows& of, const char* what) {
  if (r.N != of.N || r.H != of.H || t.scalar_type() != ref.scalar_type() || t.device() != ref.device())
    value_error(std::string(what) + " must match the rows, width, dtype (" + name_of(ref.scalar_type()) + ") and device (" +
                ref.device().str() + ") of the input");
}

// A tensor that matches the rows of `ref`.
Rows like(const Tensor& t, const Tensor& ref, const Rows& of, const char* what) {
  const Rows r = rows(t, what);
  same_rows(t, r, ref, of, what);
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

// Small outputs of one call as parts of one allocation (which costs 1.2 us of host
// time, a part 0.2): first the sizes, then the tensors.  Who keeps one keeps them all,
// so that larger ones are allocated one by one.
constexpr int64_t kSharedBytes = int64_t(1) << 20;

class Parts {
 public:
  // Reserve a tensor of `n` elements; returns its place.
  int64_t add(int64_t n, at::ScalarType t) {
    const int64_t at = bytes_;
    bytes_ += (n * (int64_t)c10::elementSize(t) + 255) / 256 * 256;
    return at;
  }
  int64_t bytes() const { return bytes_; }
  void allocate(const Tensor& ref) {
    base_ = at::empty({std::max<int64_t>(bytes_, 1)}, ref.options().dtype(at::kByte).requires_grad(false));
  }
  Tensor get(int64_t place, at::IntArrayRef sizes, at::ScalarType t) const {
    Tensor out = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base_.storage()), base_.key_set(),
                                                          at::scalarTypeToTypeMeta(t));
    out.unsafeGetTensorImpl()->set_storage_offset(place / (int64_t)c10::elementSize(t));
    out.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    return out;
  }

 private:
  Tensor base_;
  int64_t bytes_ = 0;
};

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

norm_itype tokens_of(const Tensor& tokens, const Tensor& ref, bool contiguous = true) {
  cuda_tensor(tokens, "tokens");
  const at::ScalarType t = tokens.scalar_type();
  if (t != at::kInt && t != at::kLong) type_error("tokens: dtype " + name_of(t) + " not supported (int32 or int64)");
  if (contiguous && !tokens.is_contiguous()) value_error("tokens must be contiguous");
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

// ------------------------------------------------- heads of queries and keys

// A (T, H, D) or (B, T, H, D) tensor.
struct HeadsOf {
  norm_heads h{};
  int64_t B = 1, T = 0, H = 0, D = 0;
};

HeadsOf heads_view(const Tensor& t, const char* what) {
  const int64_t d = t.dim();
  if (d != 3 && d != 4) value_error(std::string(what) + " must be (T, heads, D) or (B, T, heads, D)");
  HeadsOf r;
  if (d == 4) {
    r.B = t.size(0);
    r.h.batch_stride = t.stride(0);
  }
  r.T = t.size(d - 3);
  r.H = t.size(d - 2);
  r.D = t.size(d - 1);
  if (r.D > 1 && t.stride(d - 1) != 1) value_error(std::string(what) + ": the last dim must be contiguous");
  r.h.token_stride = t.stride(d - 3);
  r.h.head_stride = t.stride(d - 2);
  r.h.data = t.data_ptr();
  return r;
}

HeadsOf heads(const Tensor& t, const char* what) { return heads_view(cuda_tensor(t, what), what); }

// Heads of another tensor's tokens, columns, dtype and device; `H` < 0: of any number.
HeadsOf heads_like(const Tensor& t, const Tensor& ref, int64_t H, const char* what) {
  const HeadsOf r = heads(t, what);
  if (t.dim() != ref.dim() || t.scalar_type() != ref.scalar_type() || t.device() != ref.device() ||
      r.D != ref.size(-1) || r.T != ref.size(-3) || (ref.dim() == 4 && r.B != ref.size(0)) || (H >= 0 && r.H != H))
    value_error(std::string(what) + " must match the tokens, columns, heads, dtype (" + name_of(ref.scalar_type()) +
                ") and device (" + ref.device().str() + ") of what it belongs to");
  return r;
}

// cos, sin and positions; returns whether there is a rotation.
bool rotation_of(const Opt& cos, const Opt& sin, const Opt& positions, bool interleaved, const Tensor& q, const HeadsOf& of,
                 norm_rotation* r) {
  if (cos.has_value() != sin.has_value()) value_error("cos and sin come together");
  if (!cos) {
    if (positions) value_error("positions need cos and sin");
    return false;
  }
  for (const Tensor* t : {&*cos, &*sin}) {
    const char* what = t == &*cos ? "cos" : "sin";
    cuda_tensor(*t, what);
    if (t->dim() != 2 || t->sizes() != cos->sizes() || (t->size(1) > 1 && t->stride(1) != 1))
      value_error("cos and sin must be (rows, rotated columns / 2) with contiguous columns");
    if (t->device() != q.device()) value_error(std::string(what) + " is on " + t->device().str() + ", q on " + q.device().str());
    if (t->scalar_type() != cos->scalar_type()) type_error("cos and sin must share a dtype");
  }
  *r = norm_rotation{};
  r->dtype = code(cos->scalar_type(), "cos");
  if (cos->scalar_type() != q.scalar_type() && r->dtype != NORM_F32)
    type_error("cos: dtype " + name_of(cos->scalar_type()) + " must be q's or float32");
  r->rows = cos->size(0);
  r->columns = 2 * cos->size(1);
  if (r->columns < 2 || r->columns > of.D)
    value_error("cos has " + std::to_string(cos->size(1)) + " columns: 1 to " + std::to_string(of.D / 2) + " are wanted");
  r->cos = cos->data_ptr();
  r->sin = sin->data_ptr();
  r->cos_stride = r->rows > 1 ? cos->stride(0) : std::max<int64_t>(cos->size(1), 1);
  r->sin_stride = r->rows > 1 ? sin->stride(0) : std::max<int64_t>(sin->size(1), 1);
  r->interleaved = interleaved;
  if (!positions) {
    if (of.T > r->rows && of.B > 0)
      value_error(std::to_string(of.T) + " tokens a sequence, but the table has " + std::to_string(r->rows) + " rows");
    return true;
  }
  const Tensor& p = cuda_tensor(*positions, "positions");
  if (p.scalar_type() != at::kInt && p.scalar_type() != at::kLong)
    type_error("positions: dtype " + name_of(p.scalar_type()) + " not supported (int32 or int64)");
  if (p.device() != q.device()) value_error("positions are on " + p.device().str() + ", q on " + q.device().str());
  const int64_t d = p.dim();
  if (d < 1 || d > q.dim() - 2 || p.size(d - 1) != of.T || (d == 2 && p.size(0) != of.B && p.size(0) != 1))
    value_error("positions must be (T,)" + std::string(q.dim() == 4 ? " or (B, T)" : "") + ", T = " + std::to_string(of.T));
  if (of.B * of.T > 0 && r->rows == 0) value_error("the table has no rows");
  r->positions = p.data_ptr();
  r->position_type = p.scalar_type() == at::kLong ? NORM_I64 : NORM_I32;
  r->position_token_stride = p.stride(d - 1);
  r->position_batch_stride = d == 2 && p.size(0) > 1 ? p.stride(0) : 0;
  return true;
}

// Outputs shaped as q and k.  Small ones (a decode step's, where a call is host
// time) share an allocation, with the gammas' gradients if there are any; large ones
// are kept or freed one by one.
bool small(const Tensor& q, const Tensor& k) {
  return (q.numel() + k.numel()) * (int64_t)q.element_size() <= kSharedBytes;
}
struct PairPlaces {
  int64_t q, k;
  PairPlaces(Parts& parts, const Tensor& tq, const Tensor& tk)
      : q(parts.add(tq.numel(), tq.scalar_type())), k(parts.add(tk.numel(), tk.scalar_type())) {}
  void get(const Parts& parts, const Tensor& tq, const Tensor& tk, Tensor (&out)[2]) const {
    out[0] = parts.get(q, tq.sizes(), tq.scalar_type());
    out[1] = parts.get(k, tk.sizes(), tk.scalar_type());
  }
};

py::tuple head_rms_rotary_(const Tensor& q, const Opt& k, const Opt& gamma_q, const Opt& gamma_k, const Opt& cos,
                           const Opt& sin, const Opt& positions, double eps, bool interleaved, const Opt& q_out,
                           const Opt& k_out) {
  const HeadsOf qh = heads(q, "q");
  const norm_dtype xc = code(q.scalar_type(), "q");
  if (!k && (gamma_k || k_out)) value_error("gamma_k and k_out need k");
  const HeadsOf kh = k ? heads_like(*k, q, -1, "k") : HeadsOf();
  const void* gq = vec(gamma_q, qh.D, "gamma_q", q);
  const void* gk = vec(gamma_k, qh.D, "gamma_k", q);
  if (gamma_q && gamma_k && gamma_q->scalar_type() != gamma_k->scalar_type()) type_error("gamma_q and gamma_k must share a dtype");
  const norm_dtype wc = gamma_q ? code(gamma_q->scalar_type(), "gamma") : gamma_k ? code(gamma_k->scalar_type(), "gamma") : xc;
  norm_rotation rot;
  const bool turned = rotation_of(cos, sin, positions, interleaved, q, qh, &rot);
  const c10::cuda::CUDAGuard guard(q.device());
  Tensor fresh[2];
  if (!q_out && k && !k_out && small(q, *k)) {
    Parts parts;
    const PairPlaces at(parts, q, *k);
    parts.allocate(q);
    at.get(parts, q, *k, fresh);
  }
  const Tensor qo = q_out ? *q_out : fresh[0].defined() ? fresh[0] : new_like(q);
  const HeadsOf qoh = q_out ? heads_like(qo, q, qh.H, "q_out") : heads_view(qo, "q_out");
  Tensor ko;
  HeadsOf koh;
  if (k) {
    ko = k_out ? *k_out : fresh[1].defined() ? fresh[1] : new_like(*k);
    koh = k_out ? heads_like(ko, q, kh.H, "k_out") : heads_view(ko, "k_out");
  }
  if (qh.H + kh.H > 0)
    check("head_rms_rotary",
          head_rms_rotary(&qh.h, qh.H, k ? &kh.h : nullptr, kh.H, qh.H ? gq : nullptr, kh.H ? gk : nullptr, &qoh.h,
                          k ? &koh.h : nullptr, turned ? &rot : nullptr, qh.B, qh.T, qh.D, (float)eps, xc, wc, stream_of(q)));
  return py::make_tuple(obj(qo), obj(ko));
}

py::tuple head_rms_rotary_grad_(const Tensor& dyq, const Opt& dyk, const Tensor& q, const Opt& k, const Opt& gamma_q,
                                const Opt& gamma_k, const Opt& cos, const Opt& sin, const Opt& positions, double eps,
                                bool interleaved, bool need_param_grads, const Opt& workspace, const Opt& dq, const Opt& dk,
                                std::optional<at::ScalarType> param_dtype) {
  const HeadsOf qh = heads(q, "q");
  const norm_dtype xc = code(q.scalar_type(), "q");
  if (k.has_value() != dyk.has_value()) value_error("k and dyk come together");
  if (!k && (gamma_k || dk)) value_error("gamma_k and dk need k");
  const HeadsOf dyqh = heads_like(dyq, q, qh.H, "dyq");
  const HeadsOf kh = k ? heads_like(*k, q, -1, "k") : HeadsOf();
  const HeadsOf dykh = k ? heads_like(*dyk, q, kh.H, "dyk") : HeadsOf();
  const void* gq = vec(gamma_q, qh.D, "gamma_q", q);
  const void* gk = vec(gamma_k, qh.D, "gamma_k", q);
  if (gamma_q && gamma_k && gamma_q->scalar_type() != gamma_k->scalar_type()) type_error("gamma_q and gamma_k must share a dtype");
  const at::ScalarType wt = gamma_q   ? gamma_q->scalar_type()
                            : gamma_k ? gamma_k->scalar_type()
                                      : param_dtype.value_or(q.scalar_type());
  const norm_dtype wc = code(wt, "param_dtype");
  if (qh.H == 0 || (k && kh.H == 0)) value_error("q and k must have heads");
  norm_rotation rot;
  const bool turned = rotation_of(cos, sin, positions, interleaved, q, qh, &rot);
  const c10::cuda::CUDAGuard guard(q.device());
  Tensor fresh[2], dgq, dgk, ws;
  size_t wsb = 0;
  Parts parts;
  std::optional<PairPlaces> pair;
  if (!dq && k && !dk && small(q, *k)) pair.emplace(parts, q, *k);
  const int64_t at_q = need_param_grads ? parts.add(qh.D, wt) : 0, at_k = need_param_grads && k ? parts.add(qh.D, wt) : 0;
  if (pair || need_param_grads) parts.allocate(q);
  if (pair) pair->get(parts, q, *k, fresh);
  if (need_param_grads) {
    dgq = parts.get(at_q, {qh.D}, wt);
    if (k) dgk = parts.get(at_k, {qh.D}, wt);
    ws = workspace_of(workspace, head_rms_rotary_workspace_bytes(qh.D, q.get_device()), q, &wsb);
  }
  const Tensor qo = dq ? *dq : fresh[0].defined() ? fresh[0] : new_like(q);
  const HeadsOf qoh = dq ? heads_like(qo, q, qh.H, "dq") : heads_view(qo, "dq");
  Tensor ko;
  HeadsOf koh;
  if (k) {
    ko = dk ? *dk : fresh[1].defined() ? fresh[1] : new_like(*k);
    koh = dk ? heads_like(ko, q, kh.H, "dk") : heads_view(ko, "dk");
  }
  auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  check("head_rms_rotary_grad",
        head_rms_rotary_grad(&dyqh.h, &qh.h, qh.H, k ? &dykh.h : nullptr, k ? &kh.h : nullptr, kh.H, gq, gk, &qoh.h,
                             k ? &koh.h : nullptr, ptr(dgq), ptr(dgk), turned ? &rot : nullptr, ptr(ws), wsb, qh.B, qh.T,
                             qh.D, (float)eps, xc, wc, stream_of(q)));
  return py::make_tuple(obj(qo), obj(ko), obj(dgq), obj(dgk));
}

// ------------------------------------------------------ log probabilities

// The dims [result, n) of a tensor that one stride reaches; that stride, or `stride` where it is given.
int64_t flat_from(const Tensor& t, int64_t n, int64_t stride) {
  bool seen = stride != 0;
  int64_t reach = stride;
  for (int64_t i = n - 1; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (seen && t.stride(i) != reach) return i + 1;
    reach = t.size(i) * (seen ? reach : t.stride(i));
    seen = true;
  }
  return 0;
}

// Rows of logits with their tokens and their gradient as runs that one row stride
// each reaches and whose tokens are neighbours: one run where the leading dims allow
// it, else, as for logits[:, :-1] with tokens[:, 1:], one for each index of the outer
// dims, each a call of the library.
struct Runs {
  int64_t N = 0, ld = 0, ldo = 0;  // of a run
  int64_t token_size = 8;
  struct At {
    int64_t z, tok, out;  // elements from each tensor's first
  };
  c10::SmallVector<At, 1> at;
};

Runs runs_of(const Tensor& logits, const Opt& tokens, const Opt& out) {
  Runs r;
  Rows z, o;
  bool flat = row_layout(logits, "logits", &z);
  if (out) flat &= row_layout(*out, "out", &o);
  if (tokens) {
    r.token_size = tokens->element_size();
    if (tokens->numel() != z.N)
      value_error(std::to_string(z.N) + " rows of logits, but " + std::to_string(tokens->numel()) + " tokens");
  }
  const bool strided = tokens && !tokens->is_contiguous();
  if (flat && !strided) {
    r.N = z.N;
    r.ld = z.ld;
    r.ldo = o.ld;
    r.at.push_back({0, 0, 0});
    return r;
  }
  if (out && out->sizes() != logits.sizes()) value_error("out must have the logits' dims");
  const int64_t lead = logits.dim() - 1;
  const at::IntArrayRef dims = logits.sizes().slice(0, lead);
  int64_t from = flat_from(logits, lead, 0);
  if (out) from = std::max(from, flat_from(*out, lead, 0));
  if (strided) {
    if (tokens->sizes() != dims) value_error("tokens must be contiguous or of the logits' leading dims");
    if (dims[lead - 1] > 1 && tokens->stride(lead - 1) != 1)
      value_error("tokens must be contiguous along the last of the rows' dims");
    from = std::max(from, flat_from(*tokens, lead, 1));
  }
  int64_t runs = 1, inner = 0;  // the innermost dim of several rows in a run
  r.N = 1;
  for (int64_t i = 0; i < lead; ++i) {
    (i < from ? runs : r.N) *= dims[i];
    if (i >= from && dims[i] > 1) inner = i;
  }
  r.ld = r.N > 1 ? logits.stride(inner) : std::max<int64_t>(z.H, 1);
  if (out) r.ldo = r.N > 1 ? out->stride(inner) : std::max<int64_t>(z.H, 1);
  for (int64_t k = 0; k < runs; ++k) {
    Runs::At a{0, strided ? 0 : k * r.N, 0};
    for (int64_t i = from - 1, left = k; i >= 0; left /= dims[i], --i) {
      const int64_t at = left % dims[i];
      a.z += at * logits.stride(i);
      if (strided) a.tok += at * tokens->stride(i);
      if (out) a.out += at * out->stride(i);
    }
    r.at.push_back(a);
  }
  return r;
}

void* bytes_on(const void* p, int64_t bytes) { return p ? (char*)p + bytes : nullptr; }

// Where a gradient of several runs is written: the rows are distinct, and either the
// logits themselves or clear of them and of the other inputs.  (The library sees one
// run at a time.)
bool out_is_clear(const Tensor& out, const Tensor& logits, std::initializer_list<const Opt*> others) {
  struct Range {
    uintptr_t lo, hi;
  };
  auto range = [](const Tensor& t) {
    int64_t last = 0;
    for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(t.data_ptr());
    return Range{lo, lo + (uintptr_t)(last + 1) * t.element_size()};
  };
  const Range o = range(out);
  auto meets = [&](const Tensor& t) {
    const Range r = range(t);
    return o.lo < r.hi && r.lo < o.hi;
  };
  std::vector<std::pair<int64_t, int64_t>> dims;
  for (int64_t i = 0; i < out.dim(); ++i)
    if (out.size(i) > 1) dims.emplace_back(out.stride(i), out.size(i));
  std::sort(dims.begin(), dims.end());
  int64_t reach = 1;
  for (const auto& [stride, n] : dims) {
    if (stride < reach) return false;
    reach += (n - 1) * stride;
  }
  if (meets(logits) && !(out.data_ptr() == logits.data_ptr() && out.strides() == logits.strides())) return false;
  for (const Opt* t : others)
    if (*t && meets(**t)) return false;
  return true;
}

py::tuple token_logprobs_(const Tensor& logits, const Opt& tokens, double scale, int64_t top, std::optional<int64_t> ignore,
                          bool entropy) {
  Rows zr;
  row_layout(cuda_tensor(logits, "logits"), "logits", &zr);
  const norm_dtype xc = code(logits.scalar_type(), "logits");
  const norm_itype it = tokens ? tokens_of(*tokens, logits, false) : NORM_I64;
  const Runs runs = runs_of(logits, tokens, std::nullopt);
  if (top < 0 || top > NORM_MAX_TOP)
    value_error("top must be 0 to " + std::to_string(NORM_MAX_TOP) + ", not " + std::to_string(top));
  const c10::cuda::CUDAGuard guard(logits.device());
  const at::IntArrayRef lead = logits.sizes().slice(0, logits.dim() - 1);
  std::vector<int64_t> more(lead.begin(), lead.end());
  more.push_back(2);
  Parts parts;
  const int64_t a_st = parts.add(2 * zr.N, at::kFloat), a_lse = parts.add(zr.N, at::kFloat);
  const int64_t a_lp = tokens ? parts.add(zr.N, at::kFloat) : 0, a_en = entropy ? parts.add(zr.N, at::kFloat) : 0;
  const int64_t a_tlp = parts.add(zr.N * top, at::kFloat), a_tid = parts.add(zr.N * top, at::kLong);
  const bool shared = parts.bytes() <= kSharedBytes;
  if (shared) parts.allocate(logits);
  auto output = [&](int64_t place, at::IntArrayRef sizes, at::ScalarType t) {
    return shared ? parts.get(place, sizes, t) : at::empty(sizes, logits.options().dtype(t).requires_grad(false));
  };
  Tensor lp, en, tlp, tid;
  const Tensor lse = output(a_lse, lead, at::kFloat), st = output(a_st, more, at::kFloat);
  if (tokens) lp = output(a_lp, lead, at::kFloat);
  if (entropy) en = output(a_en, lead, at::kFloat);
  if (top) {
    more.back() = top;
    tlp = output(a_tlp, more, at::kFloat);
    tid = output(a_tid, more, at::kLong);
  }
  auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr<float>() : nullptr; };
  float* const p[] = {ptr(lp), ptr(en), ptr(lse), ptr(st), ptr(tlp)};
  int64_t* const ids = top ? tid.data_ptr<int64_t>() : nullptr;
  const void* const tp = tokens ? tokens->data_ptr() : nullptr;
  int64_t row = 0;
  for (const Runs::At& at : runs.at) {
    auto on = [&](float* q, int64_t n) { return q ? q + row * n : nullptr; };
    check("token_logprobs",
          token_logprobs(bytes_on(zr.p, at.z * logits.element_size()), runs.ld, bytes_on(tp, at.tok * runs.token_size), it,
                         (float)scale, ignore.value_or(NORM_NO_IGNORE), on(p[0], 1), on(p[1], 1), on(p[2], 1), on(p[3], 2),
                         on(p[4], top), ids ? ids + row * top : nullptr, top, runs.N, zr.H, xc, stream_of(logits)));
    row += runs.N;
  }
  return py::make_tuple(obj(lp), obj(en), obj(lse), obj(st), obj(tlp), obj(tid));
}

py::object token_logprobs_grad_(const Opt& dlogprob, const Tensor& logits, const Opt& tokens, const Tensor& row_stats,
                                const Opt& entropy, const Opt& dentropy, const Opt& dlse, double scale,
                                std::optional<int64_t> ignore, const Opt& out) {
  Rows zr;
  row_layout(cuda_tensor(logits, "logits"), "logits", &zr);
  const norm_dtype xc = code(logits.scalar_type(), "logits");
  const norm_itype it = tokens ? tokens_of(*tokens, logits, false) : NORM_I64;
  if (dlogprob && !tokens) value_error("dlogprob needs tokens");
  if (dentropy && !entropy) value_error("dentropy needs entropy");
  if (!dlogprob && !dentropy && !dlse) value_error("dlogprob, dentropy and dlse are all None: no gradient arrives");
  const float* dlp = stats(dlogprob, zr.N, "dlogprob", logits);
  const float* en = stats(entropy, zr.N, "entropy", logits);
  const float* den = stats(dentropy, zr.N, "dentropy", logits);
  const float* dl = stats(dlse, zr.N, "dlse", logits);
  const float* st = stats(Opt(row_stats), 2 * zr.N, "stats", logits);
  const c10::cuda::CUDAGuard guard(logits.device());
  const Tensor dz = out ? *out : new_like(logits);
  if (out) {
    Rows o;
    row_layout(cuda_tensor(dz, "out"), "out", &o);
    same_rows(dz, o, logits, zr, "out");
  }
  const Runs runs = runs_of(logits, tokens, dz);
  const Opt all_stats(row_stats);
  if (runs.at.size() > 1 && !out_is_clear(dz, logits, {&tokens, &dlogprob, &all_stats, &entropy, &dentropy, &dlse}))
    check("token_logprobs_grad", NORM_ERR_INVALID_VALUE);
  const void* const tp = tokens ? tokens->data_ptr() : nullptr;
  int64_t row = 0;
  for (const Runs::At& at : runs.at) {
    auto on = [&](const float* q, int64_t n) { return q ? q + row * n : nullptr; };
    check("token_logprobs_grad",
          token_logprobs_grad(on(dlp, 1), bytes_on(zr.p, at.z * logits.element_size()), runs.ld,
                              bytes_on(tp, at.tok * runs.token_size), it, on(st, 2), on(en, 1), on(den, 1), on(dl, 1),
                              (float)scale, ignore.value_or(NORM_NO_IGNORE), bytes_on(dz.data_ptr(), at.out * dz.element_size()),
                              runs.ldo, runs.N, zr.H, xc, stream_of(logits)));
    row += runs.N;
  }
  return obj(dz);
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
  m.def("heads_view", [](const Tensor& t) {  // (B, T, H, D, strides) of a tensor on any device, for tests
    const HeadsOf h = heads_view(t, "t");
    return py::make_tuple(h.B, h.T, h.H, h.D, h.h.batch_stride, h.h.token_stride, h.h.head_stride);
  });
  m.def("head_rms_rotary", &head_rms_rotary_);
  m.def("head_rms_rotary_grad", &head_rms_rotary_grad_);
  m.def("token_runs", [](const Tensor& logits, const Opt& tokens, const Opt& out) {  // of tensors on any device, for tests
    const Runs r = runs_of(logits, tokens, out);
    py::list at;
    for (const Runs::At& a : r.at) at.append(py::make_tuple(a.z, a.tok, a.out));
    return py::make_tuple(r.N, r.ld, at);
  });
  m.def("token_logprobs", &token_logprobs_);
  m.def("token_logprobs_grad", &token_logprobs_grad_);
}
