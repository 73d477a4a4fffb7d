// C entry points of the per-head operators (head_rms_rotary and its gradient):
// host-side validation, then dispatch to the launchers by row dtype.  Nothing is
// enqueued for an invalid call, and no entry point throws, aborts or allocates.

#include <algorithm>
#include <cmath>
#include <utility>

#include "api_common.h"
#include "common.cuh"
#include "heads.h"

using namespace normapi;
using normk::current_device_info;
using normk::DeviceInfo;
using normk::HeadArgs;
using normk::HeadView;
using normk::launch_result;

namespace {

constexpr int64_t kMaxHeads = 65535;
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1;

// A (B, T, H, D) tensor; strides of dims of one element are 0.
struct Heads {
  HeadView v{};
  int64_t B = 0, T = 0, H = 0, D = 0;
  size_t es = 1;

  // Elements from the first to the last, and one.
  int64_t extent() const { return (B - 1) * v.sb + (T - 1) * v.st + (H - 1) * v.sh + D; }
  Span span() const {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(v.p);
    return Span{lo, lo + (uint64_t)extent() * es};
  }
  // No stride negative, and the extent far inside 63 bits.
  bool in_range() const {
    const int64_t limit = (INT64_MAX / 16) / (int64_t)es;
    const int64_t n[] = {B, T, H}, s[] = {v.sb, v.st, v.sh};
    for (int i = 0; i < 3; ++i)
      if (s[i] < 0 || (n[i] > 1 && s[i] > limit / (n[i] - 1) / 4)) return false;
    return true;
  }
  // Whether no two heads share an element (enough for every layout of
  // separate dims; interleaved ones are not taken).
  bool separate() const {
    std::pair<int64_t, int64_t> d[] = {{v.sb, B}, {v.st, T}, {v.sh, H}};
    std::sort(d, d + 3);
    int64_t reach = D;
    for (const auto& [s, n] : d) {
      if (n <= 1) continue;
      if (s < reach) return false;
      reach += (n - 1) * s;
    }
    return true;
  }
};

Heads make_heads(const norm_heads* t, int64_t B, int64_t T, int64_t H, int64_t D, size_t es) {
  Heads h;
  h.v = HeadView{t->data, B > 1 ? t->batch_stride : 0, T > 1 ? t->token_stride : 0, H > 1 ? t->head_stride : 0};
  h.B = B;
  h.T = T;
  h.H = H;
  h.D = D;
  h.es = es;
  return h;
}

bool same(const Heads& a, const Heads& b) {
  return a.v.p == b.v.p && a.v.sb == b.v.sb && a.v.st == b.v.st && a.v.sh == b.v.sh && a.H == b.H;
}

// Whether two tensors of one type and of the same batches and tokens share no
// element: their ranges are apart, or they are parts of one period, as the queries
// and keys of a fused projection are: both repeat at multiples of it, and the
// columns that they take of it are apart.  The period is a token, or a batch (in
// either order, whichever is inside the other), or the least stride of all, where a
// head's query and key are side by side.  Or both have the same strides, and within
// the room of a token, whichever that is, their columns are apart.
bool apart(const Heads& a, const Heads& b) {
  if (!overlap(a.span(), b.span())) return true;
  const intptr_t bytes = (intptr_t)(reinterpret_cast<uintptr_t>(b.v.p) - reinterpret_cast<uintptr_t>(a.v.p));
  if (bytes % (intptr_t)a.es != 0) return false;
  const int64_t delta = bytes / (intptr_t)a.es;
  auto within = [&](int64_t period, int64_t wa, int64_t wb) {
    if (period <= 0) return false;
    const int64_t r = ((delta % period) + period) % period;
    return wa <= period && r >= wa && r + wb <= period;
  };
  const int64_t strides[] = {a.v.sh, a.v.st, a.v.sb, b.v.sh, b.v.st, b.v.sb};
  int64_t least = INT64_MAX;
  for (int64_t s : strides)
    if (s > 0) least = std::min(least, s);
  if (least < INT64_MAX && std::all_of(strides, strides + 6, [&](int64_t s) { return s % least == 0; }) &&
      within(least, a.D, b.D))
    return true;
  // inner and outer strides of the dims of more than one
  struct Outer {
    int64_t inner, n_inner, outer;  // outer: 0 with one such dim
  };
  auto outer = [](const Heads& h) {
    if (h.B <= 1 || h.T <= 1) return h.B > 1 ? Outer{h.v.sb, h.B, 0} : Outer{h.v.st, h.T, 0};
    return h.v.st <= h.v.sb ? Outer{h.v.st, h.T, h.v.sb} : Outer{h.v.sb, h.B, h.v.st};
  };
  const Outer oa = outer(a), ob = outer(b);
  const int64_t wa = (a.H - 1) * a.v.sh + a.D, wb = (b.H - 1) * b.v.sh + b.D;
  if (oa.inner > 0 && oa.inner == ob.inner && oa.outer % oa.inner == 0 && ob.outer % ob.inner == 0 && within(oa.inner, wa, wb))
    return true;
  if (oa.outer > 0 && oa.outer == ob.outer &&
      within(oa.outer, (oa.n_inner - 1) * oa.inner + wa, (ob.n_inner - 1) * ob.inner + wb))
    return true;
  // rooms from the first column of either to the last
  const int64_t room = std::max(wa, delta + wb) - std::min<int64_t>(0, delta);
  return a.v.sb == b.v.sb && a.v.st == b.v.st && (delta >= wa || -delta >= wb) && room <= oa.inner &&
         (oa.outer == 0 || (oa.n_inner - 1) * oa.inner + room <= oa.outer);
}

size_t index_size(norm_itype t) { return t == NORM_I64 ? 8 : 4; }

// The rotation's part of the arguments, and the ranges that it reads.
norm_status take_rotation(const norm_rotation* r, int64_t B, int64_t T, int64_t D, norm_dtype xd, HeadArgs* a, Span (&in)[3]) {
  for (Span& s : in) s = kNoSpan;
  if (r == nullptr) return NORM_OK;
  if (r->dtype != xd && r->dtype != NORM_F32) return NORM_ERR_UNSUPPORTED;
  if (r->columns < 2 || r->columns > D || r->columns % 2 != 0 || r->rows < 0) return NORM_ERR_INVALID_VALUE;
  const size_t es = elem_size(r->dtype);
  const int64_t half = r->columns / 2;
  a->R = (int)r->columns;
  a->interleaved = r->interleaved != 0;
  if (B * T == 0) return NORM_OK;
  if (!r->cos || !r->sin || !elements_aligned({r->cos, r->sin}, es) || r->rows < 1 || r->rows > (int64_t(1) << 40) ||
      !ld_ok(r->cos_stride, r->rows, half, es) || !ld_ok(r->sin_stride, r->rows, half, es))
    return NORM_ERR_INVALID_VALUE;
  in[0] = rows_span(r->cos, r->rows, r->cos_stride, half, es);
  in[1] = rows_span(r->sin, r->rows, r->sin_stride, half, es);
  if (r->positions) {
    if (r->position_type != NORM_I32 && r->position_type != NORM_I64) return NORM_ERR_UNSUPPORTED;
    if (!elements_aligned({r->positions}, index_size(r->position_type))) return NORM_ERR_INVALID_VALUE;
    Heads p;  // as heads of one element
    p.v = HeadView{const_cast<void*>(r->positions), B > 1 ? r->position_batch_stride : 0,
                   T > 1 ? r->position_token_stride : 0, 0};
    p.B = B;
    p.T = T;
    p.H = p.D = 1;
    p.es = index_size(r->position_type);
    if (!p.in_range()) return NORM_ERR_INVALID_VALUE;
    in[2] = p.span();
    a->pb = p.v.sb;
    a->pt = p.v.st;
  } else if (T > r->rows) {
    return NORM_ERR_INVALID_VALUE;  // a token would look past the table
  }
  a->cos = r->cos;
  a->ldcos = r->rows > 1 ? r->cos_stride : 0;
  a->sin = r->sin;
  a->ldsin = r->rows > 1 ? r->sin_stride : 0;
  a->table_rows = r->rows;
  a->positions = r->positions;
  a->c_f32 = r->dtype == NORM_F32;
  a->pos64 = r->position_type == NORM_I64;
  return NORM_OK;
}

template <typename F>
cudaError_t by_dtype(norm_dtype d, F&& f) {
  switch (d) {
    case NORM_BF16: return f(normk::BF16{});
    case NORM_F16: return f(normk::F16{});
    default: return f(normk::F32{});
  }
}

cudaStream_t cuda_stream(norm_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Whether a head of D columns, R of them rotated, is at most 32 units of 16: with
// halves, the rotated columns and the others are units of their own.
bool units_ok(int64_t D, const HeadArgs& a) {
  const int64_t units = a.interleaved || a.R == 0 ? (D + 15) / 16 : (a.R / 2 + 7) / 8 + (D - a.R + 15) / 16;
  return units <= 32;
}

bool sizes_ok(int64_t B, int64_t T, int64_t D, int64_t hq, int64_t hk) {
  return B >= 0 && T >= 0 && (B == 0 || T <= kMaxTokens / B) && D >= 1 && D <= normk::kHeadMaxCols && hq >= 0 &&
         hk >= 0 && hq <= kMaxHeads && hk <= kMaxHeads && hq + hk > 0;
}

size_t grad_workspace(int64_t D, const DeviceInfo& dev) {
  return std::max<size_t>(16, normk::head_grad_partials(dev) * (size_t)D * sizeof(float));
}

}  // namespace

extern "C" {

norm_status head_rms_rotary(const norm_heads* q, int64_t q_heads, const norm_heads* k, int64_t k_heads,
                            const void* gamma_q, const void* gamma_k, const norm_heads* q_out, const norm_heads* k_out,
                            const norm_rotation* rotation, int64_t B, int64_t T, int64_t D, float eps,
                            norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream) {
  NvtxRange range("head_rms_rotary");
  norm_status st = check_dtypes(x_dtype, w_dtype);
  if (st != NORM_OK) return st;
  if (!sizes_ok(B, T, D, q_heads, k_heads) || !eps_ok(eps)) return NORM_ERR_INVALID_VALUE;
  if ((q_heads == 0 && gamma_q) || (k_heads == 0 && gamma_k)) return NORM_ERR_INVALID_VALUE;
  HeadArgs a{};
  Span in[5] = {};
  {
    Span rot[3];
    st = take_rotation(rotation, B, T, D, x_dtype, &a, rot);
    if (st != NORM_OK) return st;
    if (!units_ok(D, a)) return NORM_ERR_INVALID_VALUE;
    std::copy(rot, rot + 3, in);
  }
  if (B * T == 0) return NORM_OK;
  const size_t es = elem_size(x_dtype), wes = elem_size(w_dtype);
  if (!elements_aligned({gamma_q, gamma_k}, wes)) return NORM_ERR_INVALID_VALUE;
  in[3] = gamma_q ? vec_span(gamma_q, D, wes) : kNoSpan;
  in[4] = gamma_k ? vec_span(gamma_k, D, wes) : kNoSpan;
  const norm_heads* xs[] = {q, k};
  const norm_heads* ys[] = {q_out, k_out};
  const void* gammas[] = {gamma_q, gamma_k};
  const int64_t counts[] = {q_heads, k_heads};
  Heads x[2], y[2];
  for (int i = 0; i < 2; ++i) {
    if (counts[i] == 0) continue;
    if (!xs[i] || !ys[i] || !xs[i]->data || !ys[i]->data) return NORM_ERR_INVALID_VALUE;
    x[i] = make_heads(xs[i], B, T, counts[i], D, es);
    y[i] = make_heads(ys[i], B, T, counts[i], D, es);
    if (!elements_aligned({x[i].v.p, y[i].v.p}, es) || !x[i].in_range() || !y[i].in_range() || !y[i].separate())
      return NORM_ERR_INVALID_VALUE;
    a.side[i].x = x[i].v;
    a.side[i].y = y[i].v;
    a.side[i].gamma = gammas[i];
    a.side[i].heads = (int)counts[i];
  }
  // an output may replace its own input; otherwise it is clear of the inputs and
  // of the other one
  for (int i = 0; i < 2; ++i) {
    if (counts[i] == 0) continue;
    for (int j = 0; j < 2; ++j) {
      if (counts[j] == 0) continue;
      if (!apart(y[i], x[j]) && !(i == j && same(y[i], x[j]))) return NORM_ERR_INVALID_VALUE;
      if (i < j && !apart(y[i], y[j])) return NORM_ERR_INVALID_VALUE;
    }
    const Span out[] = {y[i].span()};
    if (any_overlap(in, out)) return NORM_ERR_INVALID_VALUE;
  }
  DeviceInfo dev;
  if (!current_device_info(&dev)) return NORM_ERR_CUDA;
  a.B = B;
  a.T = T;
  a.N = B * T;
  a.D = (int)D;
  a.eps = eps;
  a.w_f32 = w_dtype == NORM_F32;
  return launch_result("head_rms_rotary launch", by_dtype(x_dtype, [&](auto d) {
                         return normk::launch_head_rotary<decltype(d)>(a, dev, cuda_stream(stream));
                       }));
}

size_t head_rms_rotary_workspace_bytes(int64_t D, int device) {
  if (D < 1 || D > normk::kHeadMaxCols) return 0;
  DeviceInfo dev;
  if (!normk::device_info_for(device, &dev)) return 0;
  return grad_workspace(D, dev);
}

norm_status head_rms_rotary_grad(const norm_heads* dyq, const norm_heads* q, int64_t q_heads, const norm_heads* dyk,
                                 const norm_heads* k, int64_t k_heads, const void* gamma_q, const void* gamma_k,
                                 const norm_heads* dq, const norm_heads* dk, void* dgamma_q, void* dgamma_k,
                                 const norm_rotation* rotation, void* workspace, size_t workspace_bytes, int64_t B,
                                 int64_t T, int64_t D, float eps, norm_dtype x_dtype, norm_dtype w_dtype,
                                 norm_stream_t stream) {
  NvtxRange range("head_rms_rotary_grad");
  norm_status st = check_dtypes(x_dtype, w_dtype);
  if (st != NORM_OK) return st;
  if (!sizes_ok(B, T, D, q_heads, k_heads) || !eps_ok(eps)) return NORM_ERR_INVALID_VALUE;
  if ((q_heads == 0 && (gamma_q || dgamma_q)) || (k_heads == 0 && (gamma_k || dgamma_k))) return NORM_ERR_INVALID_VALUE;
  const size_t es = elem_size(x_dtype), wes = elem_size(w_dtype);
  if (!elements_aligned({gamma_q, gamma_k, dgamma_q, dgamma_k}, wes)) return NORM_ERR_INVALID_VALUE;
  const Span pgrads[] = {dgamma_q ? vec_span(dgamma_q, D, wes) : kNoSpan, dgamma_k ? vec_span(dgamma_k, D, wes) : kNoSpan};
  if (overlap(pgrads[0], pgrads[1])) return NORM_ERR_INVALID_VALUE;
  HeadArgs a{};
  Span in[5] = {};
  {
    Span rot[3];
    st = take_rotation(rotation, B, T, D, x_dtype, &a, rot);
    if (st != NORM_OK) return st;
    if (!units_ok(D, a)) return NORM_ERR_INVALID_VALUE;
    std::copy(rot, rot + 3, in);
  }
  a.B = B;
  a.T = T;
  a.N = B * T;
  a.D = (int)D;
  a.eps = eps;
  a.w_f32 = w_dtype == NORM_F32;
  a.want = dgamma_q || dgamma_k;
  a.side[0].dgamma = dgamma_q;
  a.side[1].dgamma = dgamma_k;
  DeviceInfo dev;
  auto launch = [&] {
    return launch_result("head_rms_rotary_grad launch", by_dtype(x_dtype, [&](auto d) {
                           return normk::launch_head_rotary_grad<decltype(d)>(a, dev, cuda_stream(stream));
                         }));
  };
  if (a.N == 0) {
    if (!a.want) return NORM_OK;
    if (!current_device_info(&dev)) return NORM_ERR_CUDA;
    return launch();
  }
  in[3] = gamma_q ? vec_span(gamma_q, D, wes) : kNoSpan;
  in[4] = gamma_k ? vec_span(gamma_k, D, wes) : kNoSpan;
  if (any_overlap(pgrads, in)) return NORM_ERR_INVALID_VALUE;
  const norm_heads* dys[] = {dyq, dyk};
  const norm_heads* xs[] = {q, k};
  const norm_heads* dxs[] = {dq, dk};
  const void* gammas[] = {gamma_q, gamma_k};
  const int64_t counts[] = {q_heads, k_heads};
  Heads dy[2], x[2], dx[2];
  for (int i = 0; i < 2; ++i) {
    if (counts[i] == 0) continue;
    if (!dys[i] || !xs[i] || !dxs[i] || !dys[i]->data || !xs[i]->data || !dxs[i]->data) return NORM_ERR_INVALID_VALUE;
    dy[i] = make_heads(dys[i], B, T, counts[i], D, es);
    x[i] = make_heads(xs[i], B, T, counts[i], D, es);
    dx[i] = make_heads(dxs[i], B, T, counts[i], D, es);
    if (!elements_aligned({dy[i].v.p, x[i].v.p, dx[i].v.p}, es) || !dy[i].in_range() || !x[i].in_range() ||
        !dx[i].in_range() || !dx[i].separate())
      return NORM_ERR_INVALID_VALUE;
    a.side[i].x = x[i].v;
    a.side[i].y = dx[i].v;
    a.side[i].dy = dy[i].v;
    a.side[i].gamma = gammas[i];
    a.side[i].heads = (int)counts[i];
  }
  // dx may replace its own dy; otherwise outputs are clear of the inputs and of
  // each other
  for (int i = 0; i < 2; ++i) {
    if (counts[i] == 0) continue;
    for (int j = 0; j < 2; ++j) {
      if (counts[j] == 0) continue;
      if (!apart(dx[i], x[j]) || (!apart(dx[i], dy[j]) && !(i == j && same(dx[i], dy[j])))) return NORM_ERR_INVALID_VALUE;
      if (i < j && !apart(dx[i], dx[j])) return NORM_ERR_INVALID_VALUE;
    }
    const Span out[] = {dx[i].span()};
    const Span big[] = {dx[i].span(), dy[i].span(), x[i].span()};
    if (any_overlap(in, out) || any_overlap(pgrads, big)) return NORM_ERR_INVALID_VALUE;
  }
  if (a.want) {
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return NORM_ERR_WORKSPACE;
    const Span ws[] = {vec_span(workspace, (int64_t)workspace_bytes, 1)};
    if (any_overlap(ws, in) || any_overlap(ws, pgrads)) return NORM_ERR_WORKSPACE;
    for (int i = 0; i < 2; ++i) {
      if (counts[i] == 0) continue;
      const Span big[] = {dx[i].span(), dy[i].span(), x[i].span()};
      if (any_overlap(ws, big)) return NORM_ERR_WORKSPACE;
    }
  }
  if (!current_device_info(&dev)) return NORM_ERR_CUDA;
  if (a.want && workspace_bytes < grad_workspace(D, dev)) return NORM_ERR_WORKSPACE;
  a.ws = static_cast<float*>(workspace);
  return launch();
}

}  // extern "C"
