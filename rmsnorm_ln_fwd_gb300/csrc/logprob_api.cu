// C entry points of the operators at the end of a residual stream
// (token_logprobs and its gradient): host-side validation, then dispatch to the
// launchers by dtype.  Nothing is enqueued for an invalid call, and no entry
// point throws, aborts or allocates.

#include <cmath>

#include "api_common.h"
#include "common.cuh"
#include "logprob.h"

using namespace normapi;
using normk::current_device_info;
using normk::DeviceInfo;
using normk::launch_result;
using normk::LogprobArgs;
using normk::LogprobGradArgs;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 28;  // a grid of clusters of eight

template <typename F>
cudaError_t by_dtype(norm_dtype d, F&& f) {
  switch (d) {
    case NORM_BF16: return f(normk::BF16{});
    case NORM_F16: return f(normk::F16{});
    default: return f(normk::F32{});
  }
}

cudaStream_t cuda_stream(norm_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

size_t index_size(norm_itype t) { return t == NORM_I64 ? 8 : 4; }

// The scale orders the logits as they are: positive, and log2(e) times it finite.
bool scale_ok(float s) { return std::isfinite(s) && s > 0.f && std::isfinite(s * 1.4426950408889634f); }

}  // namespace

extern "C" {

norm_status token_logprobs(const void* logits, int64_t ldl, const void* tokens, norm_itype token_type, float scale,
                           int64_t ignore_index, float* logprob, float* entropy, float* lse, float* stats,
                           float* top_logprobs, int64_t* top_ids, int64_t top, int64_t N, int64_t V, norm_dtype dtype,
                           norm_stream_t stream) {
  NvtxRange range("token_logprobs");
  norm_status st = check_dtypes(dtype, dtype);
  if (st != NORM_OK) return st;
  if (tokens && token_type != NORM_I32 && token_type != NORM_I64) return NORM_ERR_UNSUPPORTED;
  if (!shape_ok(N, V) || N > kMaxRows || !scale_ok(scale) || top < 0 || top > NORM_MAX_TOP) return NORM_ERR_INVALID_VALUE;
  if (N == 0) return NORM_OK;
  const size_t es = elem_size(dtype);
  if (!logits || !ld_ok(ldl, N, V, es) || !elements_aligned({logits}, es) || (tokens == nullptr) != (logprob == nullptr) ||
      (top > 0) != (top_logprobs != nullptr) || (top > 0) != (top_ids != nullptr))
    return NORM_ERR_INVALID_VALUE;
  if (!logprob && !entropy && !lse && !stats && !top) return NORM_ERR_INVALID_VALUE;
  if (!elements_aligned({logprob, entropy, lse, top_logprobs}, 4) || !elements_aligned({stats, top_ids}, 8) ||
      (tokens && !elements_aligned({tokens}, index_size(token_type))))
    return NORM_ERR_INVALID_VALUE;
  {
    const Span in[] = {rows_span(logits, N, ldl, V, es), tokens ? vec_span(tokens, N, index_size(token_type)) : kNoSpan};
    const Span out[] = {logprob ? vec_span(logprob, N, 4) : kNoSpan, entropy ? vec_span(entropy, N, 4) : kNoSpan,
                        lse ? vec_span(lse, N, 4) : kNoSpan,         stats ? vec_span(stats, 2 * N, 4) : kNoSpan,
                        vec_span(top_logprobs, top * N, 4),          vec_span(top_ids, top * N, 8)};
    if (any_overlap(in, out)) return NORM_ERR_INVALID_VALUE;
    for (int i = 0; i < 6; ++i)
      for (int j = i + 1; j < 6; ++j)
        if (overlap(out[i], out[j])) return NORM_ERR_INVALID_VALUE;
  }
  DeviceInfo dev;
  if (!current_device_info(&dev)) return NORM_ERR_CUDA;
  LogprobArgs a{};
  a.z = logits;
  a.ldz = ldl;
  a.tokens = tokens;
  a.tok64 = token_type == NORM_I64;
  a.ignore = ignore_index;
  a.scale = scale;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.stats = reinterpret_cast<float2*>(stats);
  a.top_logprob = top_logprobs;
  a.top_id = top_ids;
  a.top = (int)top;
  a.N = N;
  a.V = (int)V;
  return launch_result("token_logprobs launch", by_dtype(dtype, [&](auto d) {
                         return normk::launch_logprob<decltype(d)>(a, dev, cuda_stream(stream));
                       }));
}

norm_status token_logprobs_grad(const float* dlogprob, const void* logits, int64_t ldl, const void* tokens,
                                norm_itype token_type, const float* stats, const float* entropy, const float* dentropy,
                                const float* dlse, float scale, int64_t ignore_index, void* dlogits, int64_t lddl,
                                int64_t N, int64_t V, norm_dtype dtype, norm_stream_t stream) {
  NvtxRange range("token_logprobs_grad");
  norm_status st = check_dtypes(dtype, dtype);
  if (st != NORM_OK) return st;
  if (dlogprob && token_type != NORM_I32 && token_type != NORM_I64) return NORM_ERR_UNSUPPORTED;
  if (!shape_ok(N, V) || N > kMaxRows || !scale_ok(scale)) return NORM_ERR_INVALID_VALUE;
  if (N == 0) return NORM_OK;
  const size_t es = elem_size(dtype);
  if (!logits || !stats || !dlogits || !ld_ok(ldl, N, V, es) || !ld_ok(lddl, N, V, es) ||
      !elements_aligned({logits, dlogits}, es) || (dlogprob && !tokens) || (dentropy && !entropy) ||
      (!dlogprob && !dentropy && !dlse))
    return NORM_ERR_INVALID_VALUE;
  if (!elements_aligned({dlogprob, entropy, dentropy, dlse}, 4) || !elements_aligned({stats}, 8) ||
      (tokens && dlogprob && !elements_aligned({tokens}, index_size(token_type))))
    return NORM_ERR_INVALID_VALUE;
  if (!same_or_disjoint(dlogits, lddl, logits, ldl, N, V, es)) return NORM_ERR_INVALID_VALUE;
  {
    const Span in[] = {dlogprob ? vec_span(dlogprob, N, 4) : kNoSpan,
                       dlogprob ? vec_span(tokens, N, index_size(token_type)) : kNoSpan,
                       vec_span(stats, 2 * N, 4),
                       dentropy ? vec_span(entropy, N, 4) : kNoSpan,
                       dentropy ? vec_span(dentropy, N, 4) : kNoSpan,
                       dlse ? vec_span(dlse, N, 4) : kNoSpan};
    const Span out[] = {rows_span(dlogits, N, lddl, V, es)};
    if (any_overlap(in, out)) return NORM_ERR_INVALID_VALUE;
  }
  DeviceInfo dev;
  if (!current_device_info(&dev)) return NORM_ERR_CUDA;
  LogprobGradArgs a{};
  a.dlogprob = dlogprob;
  a.z = logits;
  a.ldz = ldl;
  a.tokens = tokens;
  a.tok64 = token_type == NORM_I64;
  a.ignore = ignore_index;
  a.stats = reinterpret_cast<const float2*>(stats);
  a.entropy = entropy;
  a.dentropy = dentropy;
  a.dlse = dlse;
  a.scale = scale;
  a.dz = dlogits;
  a.lddz = lddl;
  a.N = N;
  a.V = (int)V;
  return launch_result("token_logprobs_grad launch", by_dtype(dtype, [&](auto d) {
                         return normk::launch_logprob_grad<decltype(d)>(a, dev, cuda_stream(stream));
                       }));
}

}  // extern "C"
