// Block join forward (sandwich_rms): the norm after a block, its gate, the
// scaled residual add and the norm before the next block, in one pass.
//
//   p = x * rstd_post * gamma_post            (or p = x)
//   h = alpha * residual + gate * p           stored, rounded to the row dtype
//   y = h * rstd_pre * gamma_pre              from the fp32 h
//   rstd = 1/sqrt(mean(v^2) + eps) of each row, fp32.
//
// A handful of flops an element: the traffic (x and residual in, h and y out)
// bounds it.

#pragma once

#include <algorithm>

#include "common.cuh"
#include "stream.h"

namespace normk {

constexpr int kJoinLoopThreads = 256;

// Any width, stride and alignment: one CTA a row at a time, a strided loop over
// the row for each of its passes (the second and third reads mostly hit L2).
// h is formed twice from the inputs, not read back, so that h_out may replace x
// or the residual: each thread has read its elements of both before it stores.
template <typename D>
__global__ void __launch_bounds__(kJoinLoopThreads) join_loop_kernel(const JoinArgs a) {
  using T = typename D::T;
  constexpr int NW = kJoinLoopThreads / 32;
  __shared__ float sh[2 * NW];
  const int lane = threadIdx.x & 31, wig = threadIdx.x >> 5;
  const bool w_f32 = a.w_f32 != 0, g_f32 = a.g_f32 != 0;
  const float inv_h = 1.f / (float)a.H;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* res = reinterpret_cast<const T*>(a.res) + row * a.ldr;
    const void* gate = a.gate;
    if (gate) gate = reinterpret_cast<const unsigned char*>(gate) + (row / a.run) * a.ldg * (g_f32 ? 4 : sizeof(T));
    float rp = 1.f;
    if (a.post) {
      float s[1] = {0.f};
      for (int j = threadIdx.x; j < a.H; j += kJoinLoopThreads) {
        const float v = load_elem<D>(x, j);
        s[0] = fmaf(v, v, s[0]);
      }
      group_sum<1>(s, sh, NW, wig, lane, 1, parity);
      parity ^= 1;
      rp = rsqrtf(s[0] * inv_h + a.eps);
      if (threadIdx.x == 0 && a.rpost) a.rpost[row] = rp;
    }
    auto stream = [&](int j) {
      float c = rp;
      if (a.post && a.gpost) c *= load_param<D>(a.gpost, j, w_f32);
      if (gate) c *= load_param<D>(gate, j, g_f32);
      return fmaf(a.alpha, load_elem<D>(res, j), c * load_elem<D>(x, j));
    };
    float rn = 0.f;
    if (a.pre) {
      float s[1] = {0.f};
      for (int j = threadIdx.x; j < a.H; j += kJoinLoopThreads) {
        const float v = stream(j);
        s[0] = fmaf(v, v, s[0]);
      }
      group_sum<1>(s, sh, NW, wig, lane, 1, parity);
      parity ^= 1;
      rn = rsqrtf(s[0] * inv_h + a.eps);
      if (threadIdx.x == 0 && a.rpre) a.rpre[row] = rn;
    }
    T* h = reinterpret_cast<T*>(a.h) + row * a.ldh;
    T* y = reinterpret_cast<T*>(a.y) + row * a.ldy;
    for (int j = threadIdx.x; j < a.H; j += kJoinLoopThreads) {
      const float v = stream(j);
      store_elem<D>(h, j, v);
      if (a.pre) store_elem<D>(y, j, v * rn * (a.gpre ? load_param<D>(a.gpre, j, w_f32) : 1.f));
    }
  }
}

template <typename D>
cudaError_t launch_join(JoinArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  const int64_t blocks = std::min<int64_t>(a.N, (int64_t)dev.sm_count * 8);
  join_loop_kernel<D><<<(unsigned)blocks, kJoinLoopThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace normk
