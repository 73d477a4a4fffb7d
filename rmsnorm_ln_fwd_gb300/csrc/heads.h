// Internal interface of the per-head operators: the RMSNorm of each head of
// queries and keys with the rotation by position (head_rms_rotary) and its
// gradient.  heads_api.cu validates the arguments; the functions here pick a
// kernel configuration and launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace normk {

constexpr int kHeadMaxCols = 512;  // 32 lanes of 16 columns

// A (B, T, H, D) tensor by its strides (elements); heads are D contiguous ones.
struct HeadView {
  void* p;
  int64_t sb, st, sh;
};

struct HeadSide {
  HeadView x;       // the heads
  HeadView y;       // forward: the output; gradient: dx
  HeadView dy;      // gradient only: the output's gradient
  const void* gamma;  // may be null (ones)
  void* dgamma;     // gradient only; may be null
  int heads;        // 0: no such side
};

struct HeadArgs {
  HeadSide side[2];  // queries, keys
  const void* cos;
  int64_t ldcos;
  const void* sin;
  int64_t ldsin;
  int64_t table_rows;
  const void* positions;  // null: token t of its sequence has position t
  int64_t pb, pt;         // position strides
  int64_t B, T, N;        // N = B * T
  int D, R;               // columns of a head; rotated ones (0: none)
  float eps;
  int w_f32;  // gammas are fp32 (else the row dtype)
  int c_f32;  // cos and sin are fp32 (else the row dtype)
  int pos64;
  int interleaved;
  unsigned* err;
  // gradient only: fp32 partial rows [CTA][side][D] of dgamma
  float* ws;
  int want;  // whether any dgamma is wanted
  // filled in by the launcher:
  int lanes;   // a head
  bool wide;   // every head starts at 16 bytes (of fp32, 32)
  int pass;    // forward: stores that leave L2 first
  int bufs;       // sets of angles a warp has
  int cvec;       // cos and sin take copies of 16 bytes
  int64_t each;   // units a warp, and how many warps have one more
  int64_t extra;
};

// Device error bit of a position outside the table.
constexpr unsigned kErrBadPosition = 8u;

// CTAs an SM, and the gradient's partial rows.
constexpr int kHeadPerSm = 2;
inline size_t head_grad_partials(const DeviceInfo& dev) { return (size_t)2 * kHeadPerSm * dev.sm_count; }

template <typename D>
cudaError_t launch_head_rotary(HeadArgs a, const DeviceInfo& dev, cudaStream_t s);
template <typename D>
cudaError_t launch_head_rotary_grad(HeadArgs a, const DeviceInfo& dev, cudaStream_t s);

}  // namespace normk
