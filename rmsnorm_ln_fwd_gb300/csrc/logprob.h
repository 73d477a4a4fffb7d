// Internal interface of the operators at the end of a residual stream: log
// probabilities of given tokens (token_logprobs) and the logits' gradient.
// logprob_api.cu validates the arguments; the functions here pick a kernel
// configuration and launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "norm.h"

namespace normk {

constexpr int kMaxTop = NORM_MAX_TOP;

struct LogprobArgs {
  const void* z;  // logits
  int64_t ldz;
  const void* tokens;  // may be null: no log probabilities
  int tok64;
  int64_t ignore;   // a token that stands for none, or NORM_NO_IGNORE
  float scale;
  float* logprob;
  float* entropy;    // may be null
  float* lse;        // may be null
  float2* stats;     // maximum and log of the sum of each row; may be null
  float* top_logprob;
  int64_t* top_id;
  int top;
  int64_t N;
  int V;
  unsigned* err;
  // filled in by the launcher:
  int cl;   // CTAs that share a row
  int tpr;  // threads a row
};

struct LogprobGradArgs {
  const float* dlogprob;  // may be null, with tokens
  const void* z;
  int64_t ldz;
  const void* tokens;
  int tok64;
  int64_t ignore;
  const float2* stats;
  const float* entropy;   // with dentropy
  const float* dentropy;  // may be null
  const float* dlse;      // may be null
  float scale;
  void* dz;
  int64_t lddz;
  int64_t N;
  int V;
  unsigned* err;
  // filled in by the launcher:
  int tx;        // threads a row
  int tiles;     // of a row
};

template <typename D>
cudaError_t launch_logprob(LogprobArgs a, const DeviceInfo& dev, cudaStream_t s);
template <typename D>
cudaError_t launch_logprob_grad(LogprobGradArgs a, const DeviceInfo& dev, cudaStream_t s);

}  // namespace normk
