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

#include "chunk.cuh"
#include "common.cuh"
#include "stream.h"

namespace normk {

constexpr int kJoinLoopThreads = 256;
constexpr float kJoinLeastEps = 1e-18f;  // (1.4e-45 / eps: 1.4e-27, under 2^-29 of eps)
// Columns a thread of the register rows: 32 bytes.
template <typename D>
constexpr int kJoinCols = 32 / (int)sizeof(typename D::T);

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

// Register rows.  A row group of tpr threads, 32 bytes of each tensor a thread
// (chunk.cuh), walks its rows with the next row's x and residual already in
// flight; gate*gamma_post and gamma_pre are products formed once (and again at
// a new gate row) in the thread's own shared-memory slot, so no barrier guards
// them.
//
// One reduction a row in place of two.  With w = gate*gamma_post and the
// reciprocal norm r of x,
//   sum(h^2) = sum((alpha*res)^2) + 2 r sum(alpha*res * w*x) + r^2 sum((w*x)^2),
// so the three sums meet in the same exchange as sum(x^2).  Where the terms
// cancel (sum(h^2) under a quarter of them) or overflow, the row takes a second
// exchange over h itself; every thread holds the same sums, so the branch is
// uniform.  So do all rows with an eps under kJoinLeastEps: squares of w*x that
// underflow (2^-149 = 1.4e-45 an element) stand for up to 1.4e-45 / eps of
// mean(h^2), which is nothing beside eps only above it.
//
// CL > 1: a cluster of CL CTAs shares each row, in parts of equal whole granules
// (the last one or two may be shorter or empty).
template <typename D, int GB, int MAXT, int MINB, int CL>
__global__ void __launch_bounds__(MAXT, MINB) join_rows_kernel(const JoinArgs a, const int tpr) {
  using C = Chunk<D, GB, kJoinCols<D>>;
  using T = typename D::T;
  constexpr int E = C::E, NP = C::NP;
  constexpr int SLOT = param_slot<E, 2>();
  extern __shared__ __align__(16) float sh_join[];
  __shared__ float xch[2][CL * 4], xch2[2][CL * 4];
  __shared__ uint64_t xbar[2], xbar2[2];
  __shared__ int xabort;
  const int rpc = blockDim.x / tpr;
  const int group = threadIdx.x / tpr;
  const int t = threadIdx.x - group * tpr;
  const int nw = tpr >> 5, wig = t >> 5, lane = threadIdx.x & 31;
  const int crank = CL > 1 ? (int)cluster_ctarank() : 0;
  // this CTA's columns [c0, c0 + H), the thread's first one c0 + b, `lim` of the
  // row's columns from there on
  const int part = CL > 1 ? ((a.H + CL * C::GE - 1) / (CL * C::GE)) * C::GE : a.H;
  const int c0 = crank * part;
  const int H = min(part, a.H - c0);  // not positive: nothing is left for this CTA
  const int b = C::base(t);
  const int lim = H - b;
  const float inv_h = 1.f / (float)a.H;
  const bool w_f32 = a.w_f32 != 0, g_f32 = a.g_f32 != 0;
  const size_t wes = w_f32 ? 4 : sizeof(T), ges = g_f32 ? 4 : sizeof(T);
  float* sh = sh_join + group * kSum4Floats;
  float* slot = sh_join + rpc * kSum4Floats + threadIdx.x * SLOT;
  const uint32_t slot32 = smem_u32(slot);
  const int bar_id = 1 + group;

  if constexpr (CL > 1) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&xbar[i], 1);
        mbar_init(&xbar2[i], 1);
      }
      xabort = 0;
      fence_barrier_init();
    }
    cluster_sync_all();  // every CTA's mbarriers exist before any CTA sends to them
  }
  pdl_launch_dependents();
  pdl_wait_primary();

  // this group's rows: strided, or (several gate rows) one contiguous range
  const int64_t units = (int64_t)(gridDim.x / CL) * rpc, unit = (int64_t)(blockIdx.x / CL) * rpc + group;
  const bool runs = a.run < a.N;
  int64_t row = unit, end = a.N, step = units;
  if (runs) {
    cta_rows(a.N, (int)unit, (int)units, row, end);
    step = 1;
  }
  uint32_t nx[C::NW], nr[C::NW];
  // Pointers that step from row to row save instructions, but not the registers
  // of three CTAs an SM (they spilled there: 8192x4096 bf16 45.9 -> 53.1 us).
  constexpr bool STEPS = MINB < 3;
  const int64_t at0 = c0 + b;
  const T* xp = reinterpret_cast<const T*>(a.x) + (STEPS ? row * a.ldx : 0) + at0;
  const T* resp = reinterpret_cast<const T*>(a.res) + (STEPS ? row * a.ldr : 0) + at0;
  T* hp = reinterpret_cast<T*>(a.h) + (STEPS ? row * a.ldh : 0) + at0;
  T* yp = reinterpret_cast<T*>(a.y) + (STEPS ? row * a.ldy : 0) + at0;
  const int64_t xstep = step * a.ldx, rstep = step * a.ldr, hstep = step * a.ldh, ystep = step * a.ldy;
  auto fetch = [&](int64_t r) {
    C::load(STEPS ? xp : xp + r * a.ldx, lim, nx);
    C::load(STEPS ? resp : resp + r * a.ldr, lim, nr);
    if constexpr (STEPS) {
      xp += xstep;
      resp += rstep;
    }
  };
  if (row < end) fetch(row);

  auto at = [](const void* p, int64_t i, size_t es) -> const void* {
    return p ? reinterpret_cast<const unsigned char*>(p) + i * es : nullptr;
  };
  int64_t gate_end = a.N;  // first row past the gate row in use
  auto stage_w = [&](int64_t r) {
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = 1.f;
    C::scale_by_param(at(a.gpost, c0, wes), w_f32, b, lim, f);
    if (a.gate) {
      const int64_t k = runs ? r / a.run : 0;
      C::scale_by_param(at(a.gate, k * a.ldg + c0, ges), g_f32, b, lim, f);
      gate_end = (k + 1) * a.run;
    }
    put_params<E>(slot, f);
  };
  if (row < end) {
    stage_w(row);
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = 1.f;
    C::scale_by_param(at(a.gpre, c0, wes), w_f32, b, lim, f);
    put_params<E>(slot + E, f);
  }

  const float2 alpha2 = splat2(a.alpha);
  int parity = 0;
  unsigned it = 0, it2 = 0;
  for (; row < end; row += step) {
    if (row >= gate_end) stage_w(row);
    float2 f[NP];     // w * x, later h
    uint32_t rw[C::NW];   // residual
#pragma unroll
    for (int k = 0; k < C::NW; ++k) rw[k] = nr[k];
    float2 sx = splat2(0.f), sa = splat2(0.f), sb = splat2(0.f), sc = splat2(0.f);
#pragma unroll
    for (int q = 0; q < NP / 2; ++q) {
      float2 w[2];
      lds_pairs(slot32 + 16 * q, w);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = 2 * q + i;
        const float2 x = word_pair<D>(nx, p);
        const float2 r = mul2(word_pair<D>(rw, p), alpha2);
        f[p] = mul2(x, w[i]);
        sx = fma2(x, x, sx);
        sa = fma2(r, r, sa);
        sb = fma2(r, f[p], sb);
        sc = fma2(f[p], f[p], sc);
      }
    }
    if (row + step < end) fetch(row + step);
    float s[4] = {sx.x + sx.y, sa.x + sa.y, sb.x + sb.y, sc.x + sc.y};
    group_sum4(s, sh, nw, wig, lane, bar_id, parity);
    parity ^= 1;
    if constexpr (CL > 1) {
      cluster_group_sum_async<4, CL>(s, xch[it & 1], &xbar[it & 1], (it >> 1) & 1u, crank, a.err, &xabort);
      ++it;
    }
    const float rp = a.post ? rsqrtf(s[0] * inv_h + a.eps) : 1.f;
    const float2 rp2 = splat2(rp);
    uint32_t out[C::NW];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      f[p] = fma2(f[p], rp2, mul2(word_pair<D>(rw, p), alpha2));
      pair_word<D>(out, p, f[p]);
    }
    C::store(STEPS ? hp : hp + row * a.ldh, lim, out);
    if constexpr (STEPS) hp += hstep;
    const bool writer = t == 0 && crank == 0;
    if (writer && a.rpost) a.rpost[row] = rp;
    if (!a.pre) continue;
    const float terms = fmaf(rp * rp, s[3], s[1]);
    float ss = fmaf(2.f * rp, s[2], terms);
    if (a.eps < kJoinLeastEps || !(ss < __int_as_float(0x7f800000)) || 4.f * ss < terms) {
      float2 h2 = splat2(0.f);
#pragma unroll
      for (int p = 0; p < NP; ++p) h2 = fma2(f[p], f[p], h2);
      float v[4] = {h2.x + h2.y, 0.f, 0.f, 0.f};
      group_sum4(v, sh, nw, wig, lane, bar_id, parity);
      parity ^= 1;
      if constexpr (CL > 1) {
        cluster_group_sum_async<1, CL>(reinterpret_cast<float(&)[1]>(v), xch2[it2 & 1], &xbar2[it2 & 1],
                                       (it2 >> 1) & 1u, crank, a.err, &xabort);
        ++it2;
      }
      ss = v[0];
    }
    const float rn = rsqrtf(ss * inv_h + a.eps);
    if (writer && a.rpre) a.rpre[row] = rn;
    const float2 rn2 = splat2(rn);
#pragma unroll
    for (int q = 0; q < NP / 2; ++q) {
      float2 g[2];
      lds_pairs(slot32 + 4 * E + 16 * q, g);
#pragma unroll
      for (int i = 0; i < 2; ++i) pair_word<D>(out, 2 * q + i, mul2(mul2(f[2 * q + i], rn2), g[i]));
    }
    C::store(STEPS ? yp : yp + row * a.ldy, lim, out);
    if constexpr (STEPS) yp += ystep;
  }
  if constexpr (CL > 1) cluster_sync_all();  // no CTA leaves while a partner may still write to it
}

template <typename D, int GB, int MAXT, int MINB, int CL>
static cudaError_t run_join_rows(const JoinArgs& a, int tpr, int rpc, const DeviceInfo& dev, cudaStream_t s) {
  auto kern = join_rows_kernel<D, GB, MAXT, MINB, CL>;
  const int threads = rpc * tpr;
  const size_t smem = sizeof(float) * ((size_t)rpc * kSum4Floats + (size_t)threads * param_slot<Chunk<D, GB, kJoinCols<D>>::E, 2>());
  static KernelMemo memo;
  if (smem > 48 * 1024) {
    cudaError_t e = memo.allow_smem(kern, dev.max_smem_optin - 1024, dev);
    if (e != cudaSuccess) return e;
  }
  const int64_t want = std::min<int64_t>((a.N + rpc - 1) / rpc, 1 << 20);
  FirstLaunch first((unsigned)threads, smem, s, CL);
  first.cfg.gridDim = dim3((unsigned)(CL * want));
  const int resident = memo.resident(threads, smem, dev, [&](int* n) {
    if (CL > 1) return cudaOccupancyMaxActiveClusters(n, kern, &first.cfg);
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, threads, smem);
    *n *= dev.sm_count;
    return e;
  });
  const int64_t grid = CL * std::max<int64_t>(1, std::min<int64_t>(want, resident));
  return first.launch((unsigned)grid, CL == 1 || grid < dev.sm_count, kern, a, tpr);
}

template <typename D, int GB>
static cudaError_t run_join(const JoinArgs& a, const DeviceInfo& dev, cudaStream_t s, bool* done) {
  *done = true;
  const int tpr = chunk_threads(a.H, kJoinCols<D>);
  // One warp a row, and fp32: three CTAs an SM; else two, which leave the
  // registers for stepping pointers (us, three; two: bf16 65536x256 29.6; 31.9,
  // 8192x1024 14.6; 13.3, 8192x4096 46.9; 47.2, 16384x4096 with eight gates 93.8;
  // 88.8, fp16 8192x2056 27.0; 24.8).
  if (tpr <= 256) {
    if constexpr (GB >= 16) {
      if (D::VEC == 4 || tpr == 32) return run_join_rows<D, GB, 256, 3, 1>(a, tpr, 256 / tpr, dev, s);
    }
    return run_join_rows<D, GB, 256, 2, 1>(a, tpr, 256 / tpr, dev, s);
  }
  // Wider rows: the smallest cluster with parts of at most 320 threads, two CTAs
  // an SM, or in fp32 256 and three (us, one CTA of up to 640 threads or
  // clusters of up to 512; 320x2; 256x3: bf16 8192x5120 56.4 as 320x2 without a
  // cluster, 6000x6144 57.6; 52.5; 64.2, 4096x8192 49.6; 50.1; 59.6, 2048x16384
  // 52.1; 52.1; 67.8, fp32 2048x8192 48.7; 48.1; 44.3, 1024x16384 51.0; 50.1;
  // 47.8).  80 registers, three CTAs of 256 threads, spill the clusters of half
  // precision.
  constexpr bool F32ROWS = D::VEC == 4;
  constexpr int T = F32ROWS ? 256 : 320, M = F32ROWS ? (GB >= 16 ? 3 : 2) : 2;
  if constexpr (!F32ROWS) {
    if (tpr <= T) return run_join_rows<D, GB, T, M, 1>(a, tpr, 1, dev, s);
  }
  auto threads = [&](int cl) {
    constexpr int GE = Chunk<D, GB, kJoinCols<D>>::GE;
    return chunk_threads((a.H + cl * GE - 1) / (cl * GE) * GE, kJoinCols<D>);
  };
  if (threads(2) <= T) return run_join_rows<D, GB, T, M, 2>(a, threads(2), 1, dev, s);
  if (threads(4) <= T) return run_join_rows<D, GB, T, M, 4>(a, threads(4), 1, dev, s);
  if (threads(8) <= T) return run_join_rows<D, GB, T, M, 8>(a, threads(8), 1, dev, s);
  *done = false;
  return cudaSuccess;
}

template <typename D>
cudaError_t launch_join(JoinArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  using T = typename D::T;
  a.err = dev.err;
  if (dev.path != PATH_LOOP) {
    GranuleRule rule;
    rule.add(a.x, a.ldx, sizeof(T));
    rule.add(a.res, a.ldr, sizeof(T));
    rule.add(a.h, a.ldh, sizeof(T));
    if (a.pre) rule.add(a.y, a.ldy, sizeof(T));
    const int gb = rule.bytes(a.H, sizeof(T));
    bool done = false;
    cudaError_t e = gb == 32   ? run_join<D, 32>(a, dev, s, &done)
                    : gb == 16 ? run_join<D, 16>(a, dev, s, &done)
                               : run_join<D, (int)sizeof(T)>(a, dev, s, &done);
    if (done) return e;
  }
  const int64_t blocks = std::min<int64_t>(a.N, (int64_t)dev.sm_count * 8);
  join_loop_kernel<D><<<(unsigned)blocks, kJoinLoopThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace normk
