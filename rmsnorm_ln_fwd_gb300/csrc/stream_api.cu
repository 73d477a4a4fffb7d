// C entry points of the residual-stream operators (the block join, its
// gradient, the token lookup and the table's gradient): host-side validation,
// then dispatch to the launchers by row dtype.  As everywhere in the library,
// nothing is enqueued for an invalid call and no entry point throws, aborts or
// allocates.

#include <algorithm>
#include <cmath>

#include "api_common.h"
#include "common.cuh"
#include "stream.h"

using namespace normapi;
using normk::current_device_info;
using normk::DeviceInfo;
using normk::JoinArgs;
using normk::JoinGradArgs;
using normk::launch_result;
using normk::LookupArgs;
using normk::LookupGradArgs;

namespace {

constexpr int64_t kMaxIds = (int64_t(1) << 31) - 2;  // table rows and tokens: 32-bit sort keys, one of them spare

template <typename F>
cudaError_t by_dtype(norm_dtype d, F&& f) {
  switch (d) {
    case NORM_BF16: return f(normk::BF16{});
    case NORM_F16: return f(normk::F16{});
    default: return f(normk::F32{});
  }
}

cudaStream_t cuda_stream(norm_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool gate_dtype_ok(norm_dtype x, norm_dtype g) { return g == x || g == NORM_F32; }

// The gate rows a call has: none without a gate, else 1 or a divisor of N.
bool gate_rows_ok(const void* gate, int64_t gate_rows, int64_t ldg, int64_t N, int64_t H, size_t ges) {
  if (gate == nullptr) return true;
  if (gate_rows < 1 || N % gate_rows != 0 || (N > 0 && gate_rows > N)) return false;
  return ld_ok(ldg, gate_rows, H, ges);
}

size_t join_workspace(int64_t H, int64_t gate_rows, const DeviceInfo& dev) {
  const size_t P = (size_t)normk::kJoinMaxPartialsPerSm * dev.sm_count;
  const size_t rows = 2 * P + (gate_rows > 1 ? 2 * P * normk::join_max_groups(H) : 0);
  return rows * (size_t)normk::bwd_partial_stride((int)H) * sizeof(float);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Two buffers of sorted pairs, the list of crossing ids, the tiles' partial
// rows: room for the tiles of any batch of up to N tokens.
size_t lookup_workspace(int64_t N, int64_t H) {
  const int64_t tiles = normk::lookup_max_tiles(N);
  return 2 * align256((size_t)N * sizeof(uint2)) + align256((size_t)(1 + tiles) * sizeof(int2)) +
         (size_t)2 * tiles * normk::bwd_partial_stride((int)H) * sizeof(float);
}

size_t index_size(norm_itype t) { return t == NORM_I64 ? 8 : 4; }

norm_status lookup_common(const void* table, int64_t ldt, int64_t V, const void* tokens, norm_itype itype,
                          const void* gamma, void* y, int64_t ldy, void* h, int64_t ldh, float* rstd, int64_t N,
                          int64_t H, float eps, float scale, bool norm, norm_dtype xd, norm_dtype wd,
                          norm_stream_t stream) {
  norm_status st = check_dtypes(xd, wd);
  if (st != NORM_OK) return st;
  if (itype != NORM_I32 && itype != NORM_I64) return NORM_ERR_UNSUPPORTED;
  if (!shape_ok(N, H) || N > kMaxIds || V < 1 || V > kMaxIds || !std::isfinite(scale)) return NORM_ERR_INVALID_VALUE;
  if (norm && !eps_ok(eps)) return NORM_ERR_INVALID_VALUE;
  if (N == 0) return NORM_OK;
  if (table == nullptr || tokens == nullptr || h == nullptr || (norm && y == nullptr)) return NORM_ERR_INVALID_VALUE;
  const size_t es = elem_size(xd);
  if (!elements_aligned({table, h, norm ? y : nullptr}, es) || !elements_aligned({gamma}, elem_size(wd)) ||
      !elements_aligned({tokens}, index_size(itype)) || !elements_aligned({rstd}, 4))
    return NORM_ERR_INVALID_VALUE;
  if (!ld_ok(ldt, V, H, es) || !ld_ok(ldh, N, H, es) || (norm && !ld_ok(ldy, N, H, es))) return NORM_ERR_INVALID_VALUE;
  {
    const Span in[] = {rows_span(table, V, ldt, H, es), vec_span(tokens, N, index_size(itype)),
                       gamma ? vec_span(gamma, H, elem_size(wd)) : kNoSpan};
    const Span rows[] = {rows_span(h, N, ldh, H, es), norm ? rows_span(y, N, ldy, H, es) : kNoSpan};
    const Span stats[] = {rstd ? vec_span(rstd, N, 4) : kNoSpan};
    if (any_overlap(in, rows) || any_overlap(in, stats) || any_overlap(rows, stats) || overlap(rows[0], rows[1]))
      return NORM_ERR_INVALID_VALUE;
  }
  DeviceInfo dev;
  if (!current_device_info(&dev)) return NORM_ERR_CUDA;
  LookupArgs a{};
  a.table = table;
  a.ldt = ldt;
  a.V = V;
  a.tokens = tokens;
  a.tok64 = itype == NORM_I64;
  a.gamma = gamma;
  a.y = norm ? y : nullptr;
  a.ldy = ldy;
  a.h = h;
  a.ldh = ldh;
  a.rstd = rstd;
  a.N = N;
  a.H = (int)H;
  a.eps = eps;
  a.scale = scale;
  a.w_f32 = wd == NORM_F32;
  return launch_result("lookup launch", by_dtype(xd, [&](auto d) {
                         return normk::launch_lookup<decltype(d)>(a, dev, cuda_stream(stream));
                       }));
}

}  // namespace

extern "C" {

norm_status sandwich_rms(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* gamma_post,
                         const void* gate, int64_t ldgate, int64_t gate_rows, const void* gamma_pre, void* y,
                         int64_t ldy, void* h_out, int64_t ldh, float* rstd_post, float* rstd_pre, int64_t N,
                         int64_t H, float eps, float residual_scale, unsigned norms, norm_dtype x_dtype,
                         norm_dtype w_dtype, norm_dtype gate_dtype, norm_stream_t stream) {
  NvtxRange range("sandwich_rms");
  norm_status st = check_dtypes(x_dtype, w_dtype);
  if (st != NORM_OK) return st;
  if (gate && !gate_dtype_ok(x_dtype, gate_dtype)) return NORM_ERR_UNSUPPORTED;
  if (!shape_ok(N, H) || !eps_ok(eps) || !std::isfinite(residual_scale)) return NORM_ERR_INVALID_VALUE;
  if ((norms & ~NORM_SANDWICH_BOTH) != 0 || norms == 0) return NORM_ERR_INVALID_VALUE;
  const bool post = norms & NORM_SANDWICH_POST, pre = norms & NORM_SANDWICH_PRE;
  // what belongs to a norm that is not taken is a mistake, not a default
  if ((!post && (gamma_post || rstd_post)) || (!pre && (gamma_pre || rstd_pre || y))) return NORM_ERR_INVALID_VALUE;
  const size_t es = elem_size(x_dtype), wes = elem_size(w_dtype), ges = elem_size(gate_dtype);
  if (!gate_rows_ok(gate, gate_rows, ldgate, N, H, ges)) return NORM_ERR_INVALID_VALUE;
  if (N == 0) return NORM_OK;
  if (!x || !residual || !h_out || (pre && !y)) return NORM_ERR_INVALID_VALUE;
  if (!elements_aligned({x, residual, h_out, y}, es) || !elements_aligned({gamma_post, gamma_pre}, wes) ||
      !elements_aligned({gate}, ges) || !elements_aligned({rstd_post, rstd_pre}, 4))
    return NORM_ERR_INVALID_VALUE;
  if (!ld_ok(ldx, N, H, es) || !ld_ok(ldr, N, H, es) || !ld_ok(ldh, N, H, es) || (pre && !ld_ok(ldy, N, H, es)))
    return NORM_ERR_INVALID_VALUE;
  if (!same_or_disjoint(h_out, ldh, x, ldx, N, H, es) || !same_or_disjoint(h_out, ldh, residual, ldr, N, H, es))
    return NORM_ERR_INVALID_VALUE;
  {
    const Span in_rows[] = {rows_span(x, N, ldx, H, es), rows_span(residual, N, ldr, H, es)};
    const Span ys[] = {pre ? rows_span(y, N, ldy, H, es) : kNoSpan};
    const Span hs[] = {rows_span(h_out, N, ldh, H, es)};
    const Span params[] = {gamma_post ? vec_span(gamma_post, H, wes) : kNoSpan,
                           gamma_pre ? vec_span(gamma_pre, H, wes) : kNoSpan,
                           gate ? rows_span(gate, gate_rows, ldgate, H, ges) : kNoSpan};
    const Span stats[] = {rstd_post ? vec_span(rstd_post, N, 4) : kNoSpan, rstd_pre ? vec_span(rstd_pre, N, 4) : kNoSpan};
    if (any_overlap(ys, in_rows) || any_overlap(ys, hs) || any_overlap(params, ys) || any_overlap(params, hs) ||
        any_overlap(params, stats) || any_overlap(stats, ys) || any_overlap(stats, hs) || any_overlap(stats, in_rows) ||
        overlap(stats[0], stats[1]))
      return NORM_ERR_INVALID_VALUE;
  }
  DeviceInfo dev;
  if (!current_device_info(&dev)) return NORM_ERR_CUDA;
  JoinArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.res = residual;
  a.ldr = ldr;
  a.gpost = gamma_post;
  a.gate = gate;
  a.ldg = ldgate;
  a.gpre = gamma_pre;
  a.y = y;
  a.ldy = ldy;
  a.h = h_out;
  a.ldh = ldh;
  a.rpost = rstd_post;
  a.rpre = rstd_pre;
  a.N = N;
  a.run = gate && gate_rows > 1 ? N / gate_rows : N;
  a.H = (int)H;
  a.eps = eps;
  a.alpha = residual_scale;
  a.post = post;
  a.pre = pre;
  a.w_f32 = w_dtype == NORM_F32;
  a.g_f32 = gate_dtype == NORM_F32;
  return launch_result("sandwich_rms launch", by_dtype(x_dtype, [&](auto d) {
                         return normk::launch_join<decltype(d)>(a, dev, cuda_stream(stream));
                       }));
}

size_t sandwich_rms_workspace_bytes(int64_t H, int64_t gate_rows, int device) {
  if (H < 1 || H > kMaxH || gate_rows < 0) return 0;
  DeviceInfo dev;
  if (!normk::device_info_for(device, &dev)) return 0;
  return join_workspace(H, gate_rows, dev);
}

norm_status sandwich_rms_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* h, int64_t ldh,
                              const float* rstd_post, const float* rstd_pre, const void* gamma_post, const void* gate,
                              int64_t ldgate, int64_t gate_rows, const void* gamma_pre, const void* dh_in,
                              int64_t lddh_in, void* dx, int64_t lddx, void* dres, int64_t lddres, void* dgamma_post,
                              void* dgate, int64_t lddgate, void* dgamma_pre, void* workspace, size_t workspace_bytes,
                              int64_t N, int64_t H, float residual_scale, unsigned norms, norm_dtype x_dtype,
                              norm_dtype w_dtype, norm_dtype gate_dtype, norm_stream_t stream) {
  NvtxRange range("sandwich_rms_grad");
  norm_status st = check_dtypes(x_dtype, w_dtype);
  if (st != NORM_OK) return st;
  if (gate && !gate_dtype_ok(x_dtype, gate_dtype)) return NORM_ERR_UNSUPPORTED;
  if (!shape_ok(N, H) || !std::isfinite(residual_scale)) return NORM_ERR_INVALID_VALUE;
  if ((norms & ~NORM_SANDWICH_BOTH) != 0 || norms == 0) return NORM_ERR_INVALID_VALUE;
  const bool post = norms & NORM_SANDWICH_POST, pre = norms & NORM_SANDWICH_PRE;
  if ((!post && (gamma_post || rstd_post || dgamma_post)) ||
      (!pre && (gamma_pre || rstd_pre || dgamma_pre || dy || h)) || (dgate && !gate))
    return NORM_ERR_INVALID_VALUE;
  const size_t es = elem_size(x_dtype), wes = elem_size(w_dtype), ges = elem_size(gate_dtype);
  if (!gate_rows_ok(gate, gate_rows, ldgate, N, H, ges)) return NORM_ERR_INVALID_VALUE;
  if (dgate && !ld_ok(lddgate, gate_rows, H, ges)) return NORM_ERR_INVALID_VALUE;
  const Span pgrads[] = {dgamma_post ? vec_span(dgamma_post, H, wes) : kNoSpan,
                         dgamma_pre ? vec_span(dgamma_pre, H, wes) : kNoSpan,
                         dgate ? rows_span(dgate, gate_rows, lddgate, H, ges) : kNoSpan};
  if (overlap(pgrads[0], pgrads[1]) || overlap(pgrads[0], pgrads[2]) || overlap(pgrads[1], pgrads[2]))
    return NORM_ERR_INVALID_VALUE;
  if (!elements_aligned({dgamma_post, dgamma_pre}, wes) || !elements_aligned({dgate}, ges)) return NORM_ERR_INVALID_VALUE;
  JoinGradArgs a{};
  a.dgpost = dgamma_post;
  a.dgate = dgate;
  a.lddg = lddgate;
  a.dgpre = dgamma_pre;
  a.N = N;
  a.H = (int)H;
  a.Hp = normk::bwd_partial_stride((int)H);
  a.w_f32 = w_dtype == NORM_F32;
  a.g_f32 = gate_dtype == NORM_F32;
  a.gate_rows = gate ? gate_rows : 0;
  a.run = N;
  auto launch = [&](const DeviceInfo& dev) {
    a.err = dev.err;
    return launch_result("sandwich_rms_grad launch", by_dtype(x_dtype, [&](auto d) {
                           return normk::launch_join_grad<decltype(d)>(a, dev, cuda_stream(stream));
                         }));
  };
  DeviceInfo dev;
  if (N == 0) {
    if (!current_device_info(&dev)) return NORM_ERR_CUDA;
    return launch(dev);
  }
  if (!x || !dx || !dres || (post && !rstd_post) || (pre && (!dy || !h || !rstd_pre)) || (!dy && !dh_in))
    return NORM_ERR_INVALID_VALUE;
  if (!elements_aligned({dy, x, h, dh_in, dx, dres}, es) || !elements_aligned({gamma_post, gamma_pre}, wes) ||
      !elements_aligned({gate}, ges) || !elements_aligned({rstd_post, rstd_pre}, 4))
    return NORM_ERR_INVALID_VALUE;
  if (!ld_ok(ldx, N, H, es) || !ld_ok(lddx, N, H, es) || !ld_ok(lddres, N, H, es) ||
      (pre && (!ld_ok(lddy, N, H, es) || !ld_ok(ldh, N, H, es))) || (dh_in && !ld_ok(lddh_in, N, H, es)))
    return NORM_ERR_INVALID_VALUE;
  // dx may replace dy and dres may replace dh_in; otherwise outputs are clear
  // of the inputs and of each other.
  const Span sdx = rows_span(dx, N, lddx, H, es), sdres = rows_span(dres, N, lddres, H, es);
  const Span sx = rows_span(x, N, ldx, H, es), sh = pre ? rows_span(h, N, ldh, H, es) : kNoSpan;
  const Span sdy = pre ? rows_span(dy, N, lddy, H, es) : kNoSpan;
  const Span sdh = dh_in ? rows_span(dh_in, N, lddh_in, H, es) : kNoSpan;
  if (overlap(sdx, sx) || overlap(sdx, sh) || overlap(sdx, sdh) || overlap(sdres, sx) || overlap(sdres, sh) ||
      overlap(sdres, sdy) || overlap(sdx, sdres) || (pre && !same_or_disjoint(dx, lddx, dy, lddy, N, H, es)) ||
      (dh_in && !same_or_disjoint(dres, lddres, dh_in, lddh_in, N, H, es)))
    return NORM_ERR_INVALID_VALUE;
  const Span small_in[] = {post ? vec_span(rstd_post, N, 4) : kNoSpan, pre ? vec_span(rstd_pre, N, 4) : kNoSpan,
                           gamma_post ? vec_span(gamma_post, H, wes) : kNoSpan,
                           gamma_pre ? vec_span(gamma_pre, H, wes) : kNoSpan,
                           gate ? rows_span(gate, gate_rows, ldgate, H, ges) : kNoSpan};
  const Span out_rows[] = {sdx, sdres};
  const Span in_rows[] = {sdy, sx, sh, sdh};
  if (any_overlap(small_in, out_rows) || any_overlap(small_in, pgrads) || any_overlap(pgrads, in_rows) ||
      any_overlap(pgrads, out_rows))
    return NORM_ERR_INVALID_VALUE;
  const bool want = dgamma_post || dgate || dgamma_pre;
  if (want) {
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return NORM_ERR_WORKSPACE;
    const Span ws[] = {vec_span(workspace, (int64_t)workspace_bytes, 1)};
    if (any_overlap(ws, small_in) || any_overlap(ws, out_rows) || any_overlap(ws, in_rows) || any_overlap(ws, pgrads))
      return NORM_ERR_WORKSPACE;
  }
  if (!current_device_info(&dev)) return NORM_ERR_CUDA;
  if (want && workspace_bytes < join_workspace(H, a.gate_rows, dev)) return NORM_ERR_WORKSPACE;
  a.dy = dy;
  a.lddy = lddy;
  a.x = x;
  a.ldx = ldx;
  a.h = h;
  a.ldh = ldh;
  a.rpost = rstd_post;
  a.rpre = rstd_pre;
  a.gpost = gamma_post;
  a.gate = gate;
  a.ldg = ldgate;
  a.gpre = gamma_pre;
  a.dh_in = dh_in;
  a.lddh = lddh_in;
  a.dx = dx;
  a.lddx = lddx;
  a.dres = dres;
  a.lddres = lddres;
  a.run = a.gate_rows > 1 ? N / a.gate_rows : N;
  a.alpha = residual_scale;
  if (want) {
    const size_t P = (size_t)normk::kJoinMaxPartialsPerSm * dev.sm_count;
    a.ws_pre = static_cast<float*>(workspace);
    a.ws_post = a.ws_pre + P * a.Hp;
    a.ws_seg = a.ws_post + P * a.Hp;
  }
  return launch(dev);
}

norm_status embedding_lookup(const void* table, int64_t ldt, int64_t V, const void* tokens, norm_itype token_type,
                             void* h, int64_t ldh, int64_t N, int64_t H, float scale, norm_dtype dtype,
                             norm_stream_t stream) {
  NvtxRange range("embedding_lookup");
  return lookup_common(table, ldt, V, tokens, token_type, nullptr, nullptr, 0, h, ldh, nullptr, N, H, 0.f, scale,
                       false, dtype, dtype, stream);
}

norm_status embedding_rms(const void* table, int64_t ldt, int64_t V, const void* tokens, norm_itype token_type,
                          const void* gamma, void* y, int64_t ldy, void* h, int64_t ldh, float* rstd, int64_t N,
                          int64_t H, float eps, float scale, norm_dtype x_dtype, norm_dtype w_dtype,
                          norm_stream_t stream) {
  NvtxRange range("embedding_rms");
  return lookup_common(table, ldt, V, tokens, token_type, gamma, y, ldy, h, ldh, rstd, N, H, eps, scale, true,
                       x_dtype, w_dtype, stream);
}

size_t embedding_grad_workspace_bytes(int64_t N, int64_t H) {
  if (N < 0 || N > kMaxIds || H < 1 || H > kMaxH) return 0;
  return std::max<size_t>(16, lookup_workspace(N, H));
}

norm_status embedding_grad(const void* dh, int64_t lddh, const void* tokens, norm_itype token_type, void* dtable,
                           int64_t lddt, int64_t V, void* workspace, size_t workspace_bytes, int64_t N, int64_t H,
                           float scale, int64_t padding_idx, int accumulate, norm_dtype x_dtype, norm_dtype w_dtype,
                           norm_stream_t stream) {
  NvtxRange range("embedding_grad");
  norm_status st = check_dtypes(x_dtype, w_dtype);
  if (st != NORM_OK) return st;
  if (token_type != NORM_I32 && token_type != NORM_I64) return NORM_ERR_UNSUPPORTED;
  if (!shape_ok(N, H) || N > kMaxIds || V < 1 || V > kMaxIds || !std::isfinite(scale) || padding_idx < -1 ||
      padding_idx >= V || dtable == nullptr)
    return NORM_ERR_INVALID_VALUE;
  const size_t es = elem_size(x_dtype), wes = elem_size(w_dtype);
  if (!ld_ok(lddt, V, H, wes) || !elements_aligned({dtable}, wes)) return NORM_ERR_INVALID_VALUE;
  LookupGradArgs a{};
  if (N > 0) {
    if (dh == nullptr || tokens == nullptr || !ld_ok(lddh, N, H, es) || !elements_aligned({dh}, es) ||
        !elements_aligned({tokens}, index_size(token_type)))
      return NORM_ERR_INVALID_VALUE;
    const Span in[] = {rows_span(dh, N, lddh, H, es), vec_span(tokens, N, index_size(token_type))};
    const Span out[] = {rows_span(dtable, V, lddt, H, wes)};
    if (any_overlap(in, out)) return NORM_ERR_INVALID_VALUE;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0 ||
        workspace_bytes < lookup_workspace(N, H))
      return NORM_ERR_WORKSPACE;
    const Span ws[] = {vec_span(workspace, (int64_t)workspace_bytes, 1)};
    if (any_overlap(ws, in) || any_overlap(ws, out)) return NORM_ERR_WORKSPACE;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    const size_t pairs = align256((size_t)N * sizeof(uint2));
    a.sorted = reinterpret_cast<uint2*>(w);
    a.other = reinterpret_cast<uint2*>(w + pairs);
    a.owners = reinterpret_cast<int2*>(w + 2 * pairs);
    a.partial = reinterpret_cast<float*>(w + 2 * pairs + align256((size_t)(1 + normk::lookup_max_tiles(N)) * sizeof(int2)));
  }
  DeviceInfo dev;
  if (!current_device_info(&dev)) return NORM_ERR_CUDA;
  a.dh = dh;
  a.lddh = lddh;
  a.tokens = tokens;
  a.tok64 = token_type == NORM_I64;
  a.dtable = dtable;
  a.lddt = lddt;
  a.V = V;
  a.N = N;
  a.H = (int)H;
  a.Hp = normk::bwd_partial_stride((int)H);
  a.scale = scale;
  a.padding = padding_idx;
  a.accumulate = accumulate != 0;
  a.w_f32 = w_dtype == NORM_F32;
  return launch_result("embedding_grad launch", by_dtype(x_dtype, [&](auto d) {
                         return normk::launch_lookup_grad<decltype(d)>(a, dev, cuda_stream(stream));
                       }));
}

}  // extern "C"
