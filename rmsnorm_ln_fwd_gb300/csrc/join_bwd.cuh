// Block join gradient (sandwich_rms_grad).
//
// With h_hat = h * rstd_pre, o_hat = x * rstd_post (or x), g = dy * gamma_pre
// and w = gate * gamma_post:
//   c     = sum(g * h_hat) / H
//   dh    = dh_in + rstd_pre * (g - h_hat * c)
//   dres  = alpha * dh
//   k     = sum(w * dh * o_hat) / H            (0 without the norm after the block)
//   dx    = rstd_post * (w * dh - o_hat * k)
//   dgamma_pre  = sum over rows of dy * h_hat
//   A           = sum over the rows of a gate row's run of dh * o_hat
//   dgate       = gamma_post * A,   dgamma_post = sum over runs of gate * A
// so one accumulator serves gate and gamma_post.
//
// One reduction a row, not two: dh is linear in c, so
//   k = [ sum(w o_hat (dh_in + rstd_pre g)) - rstd_pre c sum(w o_hat h_hat) ] / H
// and the three sums g*h_hat, w*o_hat*(dh_in + rstd_pre*g), w*o_hat*h_hat meet
// in one exchange.  Its rounding is that of sums of terms no larger than
// |w o_hat| (|dh_in| + |rstd_pre g|), the terms dh itself is formed from.
//
// Rows are split into U units.  With one gate row (or none) a unit strides over
// the rows; with several it takes a contiguous range, so that it meets each run
// once.  A run that lies inside one unit is finished there; a run that crosses
// units leaves one partial row in each (at most two a unit), which the second
// kernel sums in unit order.  The workspace is therefore bounded by the unit
// count, whatever the number of gate rows, and every sum has a fixed order.

#pragma once

#include <algorithm>

#include "common.cuh"
#include "stream.h"

namespace normk {

constexpr int kJoinGradLoopThreads = 256;

// Any width, stride and alignment: a CTA is one unit, two passes over each row.
// Column j belongs to thread j % 256, whose partial sums live in the workspace
// (plain read-modify-write, no race).
template <typename D>
__global__ void __launch_bounds__(kJoinGradLoopThreads) join_grad_loop_kernel(const JoinGradArgs a) {
  using T = typename D::T;
  constexpr int NT = kJoinGradLoopThreads;
  constexpr int NW = NT / 32;
  __shared__ float sh[2 * NW * 3];
  const int lane = threadIdx.x & 31, wig = threadIdx.x >> 5;
  const bool w_f32 = a.w_f32 != 0, g_f32 = a.g_f32 != 0;
  const float inv_h = 1.f / (float)a.H;
  const int u = blockIdx.x;
  const bool runs = a.gate_rows > 1;
  const bool want_pre = a.dgpre != nullptr, want_a = a.dgpost != nullptr || a.dgate != nullptr;
  int64_t lo, hi;
  cta_rows(a.N, u, a.U, lo, hi);
  const int64_t s_first = runs && lo < hi ? lo / a.run : 0;
  float* pre = a.ws_pre + (size_t)u * a.Hp;
  float* post = a.ws_post + (size_t)u * a.Hp;
  for (int j = threadIdx.x; j < a.H; j += NT) {
    if (want_pre) pre[j] = 0.f;
    if (want_a) post[j] = 0.f;
  }
  int parity = 0;
  int64_t seg = -1;
  for (int64_t row = lo; row < hi; ++row) {
    const int64_t g_row = runs ? row / a.run : 0;
    const void* gate = a.gate;
    if (gate) gate = reinterpret_cast<const unsigned char*>(gate) + g_row * a.ldg * (g_f32 ? 4 : sizeof(T));
    float* acc = post;  // where this row's dh * o_hat is summed
    if (runs && want_a) {
      const bool whole = g_row * a.run >= lo && (g_row + 1) * a.run <= hi;
      acc = a.ws_seg + ((size_t)2 * u + (g_row == s_first && !whole ? 0 : 1)) * a.Hp;
      if (g_row != seg) {
        for (int j = threadIdx.x; j < a.H; j += NT) acc[j] = 0.f;
        seg = g_row;
      }
    }
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* h = reinterpret_cast<const T*>(a.h) + row * a.ldh;
    const T* dy = a.dy ? reinterpret_cast<const T*>(a.dy) + row * a.lddy : nullptr;
    const T* dh_in = a.dh_in ? reinterpret_cast<const T*>(a.dh_in) + row * a.lddh : nullptr;
    const float rn = a.rpre ? a.rpre[row] : 0.f;
    const float ro = a.rpost ? a.rpost[row] : 1.f;
    struct Elem {
      float dyv, g, hh, in, oh, w;
    };
    auto load = [&](int j) {
      Elem e;
      e.dyv = dy ? load_elem<D>(dy, j) : 0.f;
      e.g = e.dyv * (dy && a.gpre ? load_param<D>(a.gpre, j, w_f32) : 1.f);
      e.hh = dy ? load_elem<D>(h, j) * rn : 0.f;
      e.in = dh_in ? load_elem<D>(dh_in, j) : 0.f;
      e.oh = load_elem<D>(x, j) * ro;
      e.w = (a.rpost && a.gpost ? load_param<D>(a.gpost, j, w_f32) : 1.f) * (gate ? load_param<D>(gate, j, g_f32) : 1.f);
      return e;
    };
    float s[3] = {0.f, 0.f, 0.f};
    for (int j = threadIdx.x; j < a.H; j += NT) {
      const Elem e = load(j);
      const float wo = e.w * e.oh;
      s[0] = fmaf(e.g, e.hh, s[0]);
      s[1] = fmaf(wo, fmaf(rn, e.g, e.in), s[1]);
      s[2] = fmaf(wo, e.hh, s[2]);
    }
    group_sum<3>(s, sh, NW, wig, lane, 1, parity);
    parity ^= 1;
    const float c = s[0] * inv_h;
    const float k = a.rpost ? fmaf(-rn * c, s[2], s[1]) * inv_h : 0.f;
    T* dx = reinterpret_cast<T*>(a.dx) + row * a.lddx;
    T* dres = reinterpret_cast<T*>(a.dres) + row * a.lddres;
    const bool last = runs && want_a && (row + 1 == hi || (row + 1) / a.run != g_row);
    const bool whole = g_row * a.run >= lo && (g_row + 1) * a.run <= hi;
    for (int j = threadIdx.x; j < a.H; j += NT) {
      const Elem e = load(j);
      const float dh = fmaf(rn, fmaf(-e.hh, c, e.g), e.in);
      store_elem<D>(dres, j, a.alpha * dh);
      store_elem<D>(dx, j, ro * fmaf(e.w, dh, -e.oh * k));
      if (want_pre) pre[j] = fmaf(e.dyv, e.hh, pre[j]);
      if (want_a) {
        const float sum = fmaf(dh, e.oh, acc[j]);
        acc[j] = sum;
        if (last) {  // the run ends here: its share of dgamma_post, and dgate if the unit holds all of it
          const float gt = load_param<D>(gate, j, g_f32);
          post[j] = fmaf(gt, sum, post[j]);
          if (whole && a.dgate) {
            const float v = sum * (a.rpost && a.gpost ? load_param<D>(a.gpost, j, w_f32) : 1.f);
            if (g_f32)
              reinterpret_cast<float*>(a.dgate)[g_row * a.lddg + j] = v;
            else
              store_elem<D>(a.dgate, g_row * a.lddg + j, v);
          }
        }
      }
    }
  }
}

// The parameter gradients from the partial rows, columns over blockIdx.x.
// blockIdx.y = 0: dgamma_pre; 1: dgamma_post (and dgate when one gate row
// serves all rows: both are products of the same sum); 2 + s: dgate of run s
// (by_boundary = 0), or of the run that crosses from unit b to b + 1 if that is
// the first boundary it crosses (by_boundary = 1, b = blockIdx.y - 2).  A CTA
// has RG row groups of 256/RG column lanes, four columns a lane; a group sums
// every RG-th partial row, then a fixed-order tree in shared memory.
constexpr int kJoinReduceUnroll = 8;

template <typename D, int RG>
__global__ void __launch_bounds__(256) join_grad_reduce_kernel(const JoinGradArgs a, int by_boundary) {
  pdl_wait_primary();  // launched as a programmatic dependent of the main kernel
  const int what = blockIdx.y;
  const float* src;
  int rows;
  int64_t ld = a.Hp, seg = 0;
  int first_slot = 0;
  if (what == 0) {
    if (a.dgpre == nullptr) return;
    src = a.ws_pre;
    rows = a.P;
  } else if (what == 1) {
    if (a.dgpost == nullptr && (a.dgate == nullptr || a.gate_rows > 1)) return;
    src = a.ws_post;
    rows = a.P;
  } else {
    // unit of row r: the largest u with floor(N*u/U) <= r
    auto unit_of = [&](int64_t r) { return (int)(((r + 1) * a.U - 1) / a.N); };
    seg = what - 2;
    if (by_boundary) {
      const int b = what - 2;
      const int64_t r = a.N * (b + 1) / a.U;  // first row of unit b + 1
      if (r % a.run == 0) return;             // a run begins there: nothing crosses
      seg = r / a.run;
      if (unit_of(seg * a.run) != b) return;  // it crossed an earlier boundary already
    }
    const int u0 = unit_of(seg * a.run), u1 = unit_of((seg + 1) * a.run - 1);
    if (u0 == u1) return;  // finished in the main kernel
    // slot 2u + 1 of the unit it begins in unless that unit begins inside it,
    // slot 2u of every later unit
    first_slot = 2 * u0 + ((a.N * u0 / a.U) / a.run == seg ? 0 : 1);
    src = a.ws_seg;
    rows = u1 - u0 + 1;
  }
  constexpr int lanes = 256 / RG;
  const int cl = threadIdx.x % lanes;
  const int rg = threadIdx.x / lanes;
  const int col = (blockIdx.x * lanes + cl) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < a.Hp) {
    for (int p0 = rg; p0 < rows; p0 += RG * kJoinReduceUnroll) {
      float4 v[kJoinReduceUnroll];
#pragma unroll
      for (int k = 0; k < kJoinReduceUnroll; ++k) {
        const int p = p0 + RG * k;
        int64_t row = p;
        if (what >= 2) row = p == 0 ? first_slot : 2 * (first_slot / 2 + p);
        v[k] = p < rows ? *reinterpret_cast<const float4*>(src + row * ld + col) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kJoinReduceUnroll; ++k) {
        acc.x += v[k].x;
        acc.y += v[k].y;
        acc.z += v[k].z;
        acc.w += v[k].w;
      }
    }
  }
  __shared__ float4 sm[256];
  sm[threadIdx.x] = acc;
  __syncthreads();
#pragma unroll
  for (int half = RG >> 1; half > 0; half >>= 1) {
    if (rg < half) {
      const float4 o = sm[threadIdx.x + half * lanes];
      float4 m = sm[threadIdx.x];
      m.x += o.x;
      m.y += o.y;
      m.z += o.z;
      m.w += o.w;
      sm[threadIdx.x] = m;
    }
    __syncthreads();
  }
  if (rg != 0) return;
  const float4 s4 = sm[threadIdx.x];
  const float vals[4] = {s4.x, s4.y, s4.z, s4.w};
  const bool w_f32 = a.w_f32 != 0, g_f32 = a.g_f32 != 0;
  auto put = [](void* out, int64_t i, float v, bool f32) {
    if (f32)
      reinterpret_cast<float*>(out)[i] = v;
    else
      store_elem<D>(out, i, v);
  };
  for (int i = 0; i < 4 && col + i < a.H; ++i) {
    const int j = col + i;
    if (what == 0) {
      put(a.dgpre, j, vals[i], w_f32);
      continue;
    }
    const float gp = a.rpost && a.gpost ? load_param<D>(a.gpost, j, w_f32) : 1.f;
    if (what == 1) {
      const float gt = a.gate && a.gate_rows <= 1 ? load_param<D>(a.gate, j, g_f32) : 1.f;
      if (a.dgpost) put(a.dgpost, j, gt * vals[i], w_f32);
      if (a.dgate && a.gate_rows <= 1) put(a.dgate, j, gp * vals[i], g_f32);
    } else {
      put(a.dgate, seg * a.lddg + j, gp * vals[i], g_f32);
    }
  }
}

template <typename D>
static cudaError_t launch_join_reduce(const JoinGradArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (a.dgpre == nullptr && a.dgpost == nullptr && a.dgate == nullptr) return cudaSuccess;
  // runs that cross units: none of one row, at most one a unit boundary
  int64_t crossing = 0;
  int by_boundary = 0;
  if (a.dgate && a.gate_rows > 1 && a.run > 1 && a.U > 1) {
    by_boundary = a.gate_rows > a.U - 1;
    crossing = by_boundary ? a.U - 1 : a.gate_rows;
  }
  const bool many = a.P > 128;
  const int cols = many ? 32 : 128;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.Hp + cols - 1) / cols), (unsigned)(2 + crossing));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = many ? cudaLaunchKernelEx(&cfg, join_grad_reduce_kernel<D, 32>, a, by_boundary)
                       : cudaLaunchKernelEx(&cfg, join_grad_reduce_kernel<D, 8>, a, by_boundary);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// A sum over no rows: the parameter gradients are zero.
template <typename D>
__global__ void join_grad_zero_kernel(const JoinGradArgs a) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.H) return;
  auto zero = [&](void* p, int64_t at, bool f32) {
    if (f32)
      reinterpret_cast<float*>(p)[at] = 0.f;
    else
      store_elem<D>(p, at, 0.f);
  };
  if (a.dgpre) zero(a.dgpre, i, a.w_f32);
  if (a.dgpost) zero(a.dgpost, i, a.w_f32);
  if (a.dgate)
    for (int64_t g = 0; g < a.gate_rows; ++g) zero(a.dgate, g * a.lddg + i, a.g_f32);
}

template <typename D>
cudaError_t launch_join_grad(JoinGradArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  if (a.N == 0) {
    if (a.dgpre == nullptr && a.dgpost == nullptr && a.dgate == nullptr) return cudaSuccess;
    join_grad_zero_kernel<D><<<(unsigned)((a.H + 255) / 256), 256, 0, s>>>(a);
    return cudaGetLastError();
  }
  const int cap = kJoinMaxPartialsPerSm * dev.sm_count;
  a.P = a.U = (int)std::min<int64_t>(a.N, cap);
  join_grad_loop_kernel<D><<<(unsigned)a.P, kJoinGradLoopThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join_reduce<D>(a, dev, s);
}

}  // namespace normk
