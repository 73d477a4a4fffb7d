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

#include "chunk.cuh"
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
      store_elem<D>(dx, j, a.rpost ? ro * fmaf(e.w, dh, -e.oh * k) : e.w * dh);
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

// Rows through shared memory.  A row group of tpr threads, E columns a thread
// (chunk.cuh), takes its rows from a ring of NB row buffers of its own: lanes
// 8k (k = 0..3) of its first warp bulk-copy the next row of dy, dh_in, h and x
// into a buffer, completing on its mbarrier, when the row sums' barrier has
// passed (every thread has then read the buffer).  The four lanes issue
// together: one thread issuing all four kept its warp, and with it the row
// sums' barrier, behind (barrier stalls 2.8 a cycle issued).  No registers hold
// a row in flight, and between its two passes a row waits in them as it was
// read, packed.  That leaves room for the two accumulators (dgamma_pre, and A
// for gate and gamma_post) of sixteen columns a thread, over which the work a
// row costs whatever its width (waits, row sums, addresses: half the
// instructions at eight columns) is spread.  Shared memory is read 16
// bytes a lane, a warp's reads contiguous, whatever the rows' alignment.
//
// Rows that are not 16-byte aligned (GB = one element): the copy takes the
// whole 16-byte lines inside the row; the up to 15 bytes at either end come by
// ordinary loads of the group's first warp, issued with the copy (lane 8k + i
// takes element i of both ends of tensor k) and put into the buffer a row later.
//
// CL > 1: a cluster of CL CTAs shares each row in parts of equal whole granules;
// the row sums meet through distributed shared memory.
constexpr int kJoinRowTensors = 4;  // dy, dh_in, h, x
constexpr int kJoinMaxBuffers = 4;  // row buffers a group
constexpr int kJoinMinBuffers = 2;
constexpr int kJoinMaxGroups = 8;
// Columns a thread.
template <typename D>
constexpr int kJoinGradCols = D::VEC == 8 ? 16 : 8;
constexpr int kJoinRedStride = 24;  // warps of a group, at most
constexpr int kJoinRedFloats = 2 * 3 * kJoinRedStride;

struct JoinRing {
  int tpr, rpc, nb;
  int part;        // columns a CTA of the cluster takes
  int buf_bytes;   // of one tensor's part of a row
  int red_off, par_off, buf_off, total;
};

// Shared memory: [mbarriers][abort flag][where in its 16-byte line each
// tensor's row of each buffer starts][row sums][parameters][rows].
constexpr int kJoinBarBytes = kJoinMaxGroups * kJoinMaxBuffers * 8;
constexpr int kJoinAbortOff = kJoinBarBytes;
constexpr int kJoinShiftOff = kJoinAbortOff + 16;
constexpr int kJoinRedOff = kJoinShiftOff + kJoinMaxGroups * kJoinMaxBuffers * kJoinRowTensors * 4;

constexpr int kJoinStaticSmem = 512;  // of the kernel's own, at most

// The ring of a CTA of at most `threads` threads, `ctas` of them an SM.  Several
// gate rows (`runs`) hold a third vector a thread beside its two parameters, the
// share of dgamma_post of the runs that have ended.
template <int E>
inline JoinRing join_ring(int H, int es, int ge, int cl, bool runs, int threads, int ctas, int max_smem) {
  JoinRing r{};
  r.part = (H + cl * ge - 1) / (cl * ge) * ge;
  r.tpr = chunk_threads(r.part, E);
  r.rpc = cl == 1 && r.tpr <= threads ? std::min(threads / r.tpr, kJoinMaxGroups) : 1;
  r.buf_bytes = (r.part * es + (ge * es < 16 ? 16 : 0) + 15) & ~15;
  r.red_off = kJoinRedOff;
  r.par_off = r.red_off + r.rpc * kJoinRedFloats * 4;
  const int slot = runs ? param_slot<E, 3>() : param_slot<E, 2>();
  r.buf_off = (r.par_off + r.rpc * r.tpr * slot * 4 + 127) & ~127;
  const int stage = r.rpc * kJoinRowTensors * r.buf_bytes;
  r.nb = std::min(kJoinMaxBuffers, ((max_smem + 1024) / ctas - 1024 - kJoinStaticSmem - r.buf_off) / stage);
  const int fold = r.rpc > 1 ? r.rpc * r.tpr * E * 4 : 0;  // the groups' accumulators, after the rows
  r.total = r.buf_off + std::max(r.nb * stage, fold);
  return r;
}

// The rows of unit u: the first, how many, and the distance between them.
template <bool RUNS>
__device__ __forceinline__ void join_unit_rows(const JoinGradArgs& a, int u, int64_t units, int64_t& first, int64_t& n,
                                               int64_t& step) {
  if (RUNS) {
    int64_t hi = 0;
    first = 0;
    if (u < a.U) cta_rows(a.N, u, a.U, first, hi);
    n = hi - first;
    step = 1;
  } else {
    first = u;
    step = units;
    n = u < a.N ? (a.N - u + units - 1) / units : 0;
  }
}

template <typename D, int GB, bool RUNS, int MAXT, int MINB, int CL>
__global__ void __launch_bounds__(MAXT, MINB) join_grad_rows_kernel(const JoinGradArgs a, const JoinRing ring) {
  using C = Chunk<D, GB, kJoinGradCols<D>>;
  using T = typename D::T;
  constexpr int E = C::E, NP = C::NP, NW = C::NW, ES = C::ES;
  constexpr bool EDGES = GB < 16;
  constexpr int SLOT = param_slot<E, RUNS ? 3 : 2>();
  extern __shared__ __align__(128) unsigned char sm_join[];
  __shared__ float xch[2][CL * 4];
  __shared__ uint64_t xbar[2];
  const int tpr = ring.tpr;
  const int crank = CL > 1 ? (int)cluster_ctarank() : 0;
  const int c0 = crank * ring.part;
  const int H = min(ring.part, a.H - c0);  // this CTA's columns (not positive: none)
  const int64_t units = (int64_t)(gridDim.x / CL) * ring.rpc;
  const int unit0 = ((int)blockIdx.x / CL) * ring.rpc;
  const bool copies = H > 0;

  if (threadIdx.x < kJoinMaxGroups * kJoinMaxBuffers) {
    mbar_init(reinterpret_cast<uint64_t*>(sm_join) + threadIdx.x, kJoinRowTensors);
    if (threadIdx.x == 0) {
      *reinterpret_cast<volatile int*>(sm_join + kJoinAbortOff) = 0;
      mbar_init(&xbar[0], 1);
      mbar_init(&xbar[1], 1);
    }
    fence_barrier_init();
  }
  __syncthreads();

  const int group = threadIdx.x / tpr;
  const int t = threadIdx.x - group * tpr;
  const int nw = tpr >> 5, wig = t >> 5, lane = threadIdx.x & 31;
  const int b0 = C::base(t);
  const int lim = H - b0;
  const float inv_h = 1.f / (float)a.H;
  const bool w_f32 = a.w_f32 != 0, g_f32 = a.g_f32 != 0;
  const size_t wes = w_f32 ? 4 : sizeof(T), ges = g_f32 ? 4 : sizeof(T);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm_join) + group * kJoinMaxBuffers;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm_join + kJoinAbortOff);
  float* red = reinterpret_cast<float*>(sm_join + ring.red_off) + group * kJoinRedFloats;
  float* slot = reinterpret_cast<float*>(sm_join + ring.par_off) + threadIdx.x * SLOT;
  const int row_bytes = kJoinRowTensors * ring.buf_bytes;  // a row's four buffers
  unsigned char* bufs = sm_join + ring.buf_off + (size_t)group * ring.nb * row_bytes;
  const int bar_id = 1 + group;
  const int NB = ring.nb;
  const bool has_dy = a.dy != nullptr && copies, has_in = a.dh_in != nullptr && copies;
  int* shift = reinterpret_cast<int*>(sm_join + kJoinShiftOff) + group * kJoinMaxBuffers * kJoinRowTensors;

  const int unit = unit0 + group;
  int64_t row, step, left;
  join_unit_rows<RUNS>(a, unit, units, row, left, step);
  const int64_t first_row = row, end = row + left * step;  // (RUNS: step is 1)

  if (a.early) pdl_launch_dependents();
  pdl_wait_primary();

  // Copies: lane 8k + i of the group's first warp serves tensor k.
  const int ck = lane >> 3, ci = lane & 7;
  const T* next = nullptr;  // the tensor's next row to ask for
  int64_t next_step = 0;
  if (wig == 0 && copies) {
    next = reinterpret_cast<const T*>(ck == 0 ? a.dy : ck == 1 ? a.dh_in : ck == 2 ? (has_dy ? a.h : nullptr) : a.x);
    next_step = step * (ck == 0 ? a.lddy : ck == 1 ? a.lddh : ck == 2 ? a.ldh : a.ldx);
    if (next) next += row * (ck == 0 ? a.lddy : ck == 1 ? a.lddh : ck == 2 ? a.ldh : a.ldx) + c0;
  }
  int issued = 0;  // rows asked for
  T edge0 = T(0.f), edge1 = T(0.f);
  int edge_at0 = -1, edge_at1 = -1;  // byte offsets in the row buffers, or none
  auto issue = [&](int buf) {  // by the group's first warp
    const uintptr_t s = reinterpret_cast<uintptr_t>(next), e = s + (uintptr_t)H * ES, line = s & ~(uintptr_t)15;
    const uintptr_t up = (s + 15) & ~(uintptr_t)15, down = e & ~(uintptr_t)15;
    const int dst = buf * row_bytes + ck * ring.buf_bytes;
    if constexpr (EDGES) {
      edge_at0 = edge_at1 = -1;
      if (next) {
        // front [s, min(up, e)), back [max(up, down), e): at most 8 elements each
        const uintptr_t p0 = s + (uintptr_t)ci * ES, p1 = (down > up ? down : up) + (uintptr_t)ci * ES;
        if (p0 < (up < e ? up : e)) {
          edge0 = *reinterpret_cast<const T*>(p0);
          edge_at0 = dst + (int)(p0 - line);
        }
        if (p1 < e) {
          edge1 = *reinterpret_cast<const T*>(p1);
          edge_at1 = dst + (int)(p1 - line);
        }
      }
    }
    if (ci == 0) {
      const uint32_t n = next && down > up ? (uint32_t)(down - up) : 0u;
      if constexpr (EDGES) shift[buf * kJoinRowTensors + ck] = (int)(s - line);
      mbar_arrive_expect_tx(&full[buf], n);
      if (n != 0) bulk_g2s(bufs + dst + (up - line), reinterpret_cast<const void*>(up), n, &full[buf]);
    }
    if (next) next += next_step;
    ++issued;
  };
  auto edge_store = [&]() {
    if constexpr (EDGES) {
      if (edge_at0 >= 0) *reinterpret_cast<T*>(bufs + edge_at0) = edge0;
      if (edge_at1 >= 0) *reinterpret_cast<T*>(bufs + edge_at1) = edge1;
      edge_at0 = edge_at1 = -1;
    }
  };
  if (wig == 0 && copies) {
    for (int i = 0; i < NB && i < left; ++i) {
      issue(i);
      edge_store();
    }
  }

  auto at = [](const void* p, int64_t i, size_t es) -> const void* {
    return p ? reinterpret_cast<const unsigned char*>(p) + i * es : nullptr;
  };
  int64_t gate_row = 0, gate_end = a.N;
  auto stage_w = [&](int64_t r) {
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = 1.f;
    C::scale_by_param(a.rpost ? at(a.gpost, c0, wes) : nullptr, w_f32, b0, lim, f);
    if (a.gate) {
      gate_row = RUNS ? r / a.run : 0;
      gate_end = (gate_row + 1) * a.run;
      C::scale_by_param(at(a.gate, gate_row * a.ldg + c0, ges), g_f32, b0, lim, f);
    }
    put_params<E>(slot, f);
  };
  {
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = 1.f;
    C::scale_by_param(at(a.gpre, c0, wes), w_f32, b0, lim, f);
    put_params<E>(slot + E, f);
    if (left > 0) stage_w(row);
    if constexpr (RUNS) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = 0.f;
      put_params<E>(slot + 2 * E, f);
    }
  }
  if constexpr (EDGES) named_barrier(bar_id, tpr);  // the first rows' ends are in place
  if constexpr (CL > 1) cluster_sync_all();         // every CTA's mbarriers exist before any CTA sends to them

  float2 acc_pre[NP], acc[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) acc_pre[p] = acc[p] = splat2(0.f);

  // A run ends (RUNS): its share of dgamma_post, and dgate if it lies in this
  // unit, else a partial row.
  auto flush = [&](int64_t k) {
    if constexpr (RUNS) {
      const bool whole = k * a.run >= first_row && (k + 1) * a.run <= end;
      const int64_t part_row = 2 * (int64_t)unit + (!whole && k == first_row / a.run ? 0 : 1);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = c0 + b0 + C::col(e);
        if (C::col(e) < lim) {
          const float v = (e & 1) ? acc[e / 2].y : acc[e / 2].x;
          slot[2 * E + e] = fmaf(load_param<D>(at(a.gate, k * a.ldg, ges), c, g_f32), v, slot[2 * E + e]);
          if (!whole) {
            if (a.ws_seg) a.ws_seg[part_row * a.Hp + c] = v;
          } else if (a.dgate) {
            const float g = v * (a.rpost && a.gpost ? load_param<D>(a.gpost, c, w_f32) : 1.f);
            if (g_f32)
              reinterpret_cast<float*>(a.dgate)[k * a.lddg + c] = g;
            else
              store_elem<D>(a.dgate, k * a.lddg + c, g);
          }
        }
      }
#pragma unroll
      for (int p = 0; p < NP; ++p) acc[p] = splat2(0.f);
    }
  };

  T* dxp = reinterpret_cast<T*>(a.dx) + row * a.lddx + c0 + b0;
  T* drp = reinterpret_cast<T*>(a.dres) + row * a.lddres + c0 + b0;
  const int64_t dx_step = step * a.lddx, dr_step = step * a.lddres;
  // The thread's columns of tensor k, from a row buffer.
  const uint32_t bufs32 = smem_u32(bufs) + b0 * ES, slot32 = smem_u32(slot);
  auto read = [&](uint32_t p, bool there, uint32_t (&w)[NW]) {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = 0u;
    if (!there) return;
    if constexpr (GB >= 16) {
#pragma unroll
      for (int g = 0; g < C::NG; ++g)
        if (C::col(g * C::GE) < lim) lds_words<4>(p + C::col(g * C::GE) * ES, w + 4 * g);
    } else if constexpr (ES == 4) {
#pragma unroll
      for (int g = 0; g < C::NG; ++g)
        if (C::col(g) < lim) w[g] = lds_u32(p + C::col(g) * 4);
    } else {
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const uint32_t lo = C::col(2 * i) < lim ? lds_u16(p + C::col(2 * i) * 2) : 0u;
        const uint32_t hi = C::col(2 * i + 1) < lim ? lds_u16(p + C::col(2 * i + 1) * 2) : 0u;
        w[i] = __byte_perm(lo, hi, 0x5410);
      }
    }
  };
  const float2 alpha2 = splat2(a.alpha);
  const bool post = a.rpost != nullptr;
  int parity = 0, buf = 0;
  unsigned phase = 0u, it = 0;  // phase: parity of the ring's current turn
  float nrn = 0.f, nro = 1.f;   // the next row's statistics
  auto fetch_stats = [&](int64_t r) {
    if (a.rpre) nrn = a.rpre[r];
    if (a.rpost) nro = a.rpost[r];
  };
  if (left > 0) fetch_stats(row);
  for (; left > 0; --left, row += step) {
    if (RUNS && row >= gate_end) {
      flush(gate_row);
      stage_w(row);
    }
    const float rn = nrn, ro = nro;
    if (left > 1) fetch_stats(row + step);
    edge_store();
    int ok = 1;
    if (copies) ok = mbar_wait(&full[buf], phase, a.err, abort_flag);
    asm volatile("" : "+r"(ok));  // one body for both outcomes
    uint32_t dyw[NW], iw[NW], hw[NW], xw[NW];
    {
      const uint32_t base = bufs32 + buf * row_bytes;
      const int* sft = shift + buf * kJoinRowTensors;
      read(base + (EDGES ? sft[0] : 0), has_dy, dyw);
      read(base + ring.buf_bytes + (EDGES ? sft[1] : 0), has_in, iw);
      read(base + 2 * ring.buf_bytes + (EDGES ? sft[2] : 0), has_dy, hw);
      read(base + 3 * ring.buf_bytes + (EDGES ? sft[3] : 0), copies, xw);
    }
    // pass 1: the row's three sums over t = dh_in + rstd_pre * g, h and x (the
    // statistics that turn h and x into h_hat and o_hat come in behind)
    float s[3];
    {
      float2 s0 = splat2(0.f), s1 = splat2(0.f), s2 = splat2(0.f);
      const float2 rn2 = splat2(rn);
#pragma unroll
      for (int q = 0; q < NP / 2; ++q) {
        float2 w[2], gp[2];
        lds_pairs(slot32 + 16 * q, w);
        lds_pairs(slot32 + 4 * E + 16 * q, gp);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int p = 2 * q + i;
          const float2 g = mul2(word_pair<D>(dyw, p), gp[i]);
          const float2 wx = mul2(word_pair<D>(xw, p), w[i]);
          const float2 h = word_pair<D>(hw, p);
          s0 = fma2(g, h, s0);
          s1 = fma2(wx, fma2(g, rn2, word_pair<D>(iw, p)), s1);
          s2 = fma2(wx, h, s2);
        }
      }
      s[0] = s0.x + s0.y;
      s[1] = s1.x + s1.y;
      s[2] = s2.x + s2.y;
    }
    {
      // value k in lanes 8k..8k+7 of each warp, then eight lanes a value over the group's warps
      float part = warp_sum_scatter<3>(s, lane);
      if (nw > 1) {
        const int v = min(lane >> 3, 2);
        if ((lane & 7) == 0 && lane < 24) red[(parity * 3 + v) * kJoinRedStride + wig] = part;
        named_barrier(bar_id, tpr);
        const float* from = red + (parity * 3 + v) * kJoinRedStride;
        part = 0.f;
#pragma unroll
        for (int i = 0; i < kJoinRedStride / 8; ++i)
          if ((lane & 7) + 8 * i < nw) part += from[(lane & 7) + 8 * i];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      } else {
        // one warp: what the barrier orders besides the sums, its lanes' reads of
        // this buffer before the refill and the end elements put into the others
        // before their reads (shuffles order no memory)
        __syncwarp();
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) s[k] = __shfl_sync(0xffffffffu, part, 8 * k);
    }
    parity ^= 1;
    // every thread has read this buffer: refill it with the row NB ahead
    if (wig == 0 && copies && left > NB && !*abort_flag) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      issue(buf);
    }
    if constexpr (CL > 1) {
      ok &= (int)cluster_group_sum_async<3, CL>(s, xch[it & 1], &xbar[it & 1], (it >> 1) & 1u, crank, a.err, abort_flag);
      ++it;
    }
    // c = mean(g h_hat), dh = t - rstd_pre c h_hat, k = mean(w dh o_hat)
    const float crr = s[0] * inv_h * rn * rn * rn;
    const float k = a.rpost ? ro * fmaf(-crr, s[2], s[1]) * inv_h : 0.f;
    const float2 nc2 = splat2(-crr), rn2 = splat2(rn), ro2 = splat2(ro), nk2 = splat2(-k * ro * ro);
    uint32_t od[NW], ox[NW];
    // Unpack again rather than hold the fp32 values over the barrier.  The wait
    // (for the phase before a barrier's first: over before it begins) is there
    // for the compiler, which otherwise moves the outputs' unpacking up among
    // the row sums and spills 184 bytes a thread; a cluster has one of its own.
    if constexpr (CL == 1) mbar_wait(&xbar[0], 1u, a.err, nullptr);
#pragma unroll
    for (int i = 0; i < NW; ++i) asm volatile("" : "+r"(dyw[i]), "+r"(iw[i]), "+r"(hw[i]), "+r"(xw[i]));
#pragma unroll
    for (int q = 0; q < NP / 2; ++q) {
      float2 w[2], gp[2];
      lds_pairs(slot32 + 16 * q, w);
      lds_pairs(slot32 + 4 * E + 16 * q, gp);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = 2 * q + i;
        const float2 x = word_pair<D>(xw, p), h = word_pair<D>(hw, p);
        const float2 dyr = mul2(word_pair<D>(dyw, p), rn2);
        const float2 dh = fma2(h, nc2, fma2(dyr, gp[i], word_pair<D>(iw, p)));
        pair_word<D>(od, p, mul2(dh, alpha2));
        const float2 dr = mul2(dh, ro2);
        float2 o = mul2(dr, w[i]);
        if (post) o = fma2(x, nk2, o);  // (0 times an infinite x is no 0)
        pair_word<D>(ox, p, o);
        acc_pre[p] = fma2(dyr, h, acc_pre[p]);
        acc[p] = fma2(dr, x, acc[p]);
      }
    }
    if (ok) {
      C::store(drp, lim, od);
      C::store(dxp, lim, ox);
    }
    drp += dr_step;
    dxp += dx_step;
    if (++buf == NB) {
      buf = 0;
      phase ^= 1u;
    }
  }
  if (t == 0)  // no copy outlives the CTA (they have all been waited for unless a wait ran out)
    for (int q = 0; q < NB && q < issued; ++q) mbar_wait(&full[q], (unsigned)((issued - 1 - q) / NB) & 1u, a.err, nullptr);
  if (RUNS && first_row < end) flush(gate_row);
  if constexpr (CL > 1) cluster_sync_all();  // no CTA leaves while a partner may still write to it
  if (a.ws_pre == nullptr) return;
  if constexpr (RUNS) {
#pragma unroll
    for (int p = 0; p < NP; ++p) acc[p] = make_float2(slot[2 * E + 2 * p], slot[2 * E + 2 * p + 1]);
  }
  // The CTA's partial rows: its groups' accumulators in group order.
  const int prow = (int)blockIdx.x / CL;
  auto partial = [&](float2 (&v)[NP], float* ws) {
    if (ring.rpc > 1) {
      float* fold = reinterpret_cast<float*>(sm_join + ring.buf_off);
      __syncthreads();
#pragma unroll
      for (int q = 0; q < NP / 2; ++q)
        *reinterpret_cast<float4*>(fold + ((size_t)q * blockDim.x + threadIdx.x) * 4) =
            make_float4(v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y);
      __syncthreads();
      if (group != 0) return;
      for (int g = 1; g < ring.rpc; ++g) {
#pragma unroll
        for (int q = 0; q < NP / 2; ++q) {
          const float4 o = *reinterpret_cast<const float4*>(fold + ((size_t)q * blockDim.x + g * tpr + t) * 4);
          v[2 * q] = add2(v[2 * q], make_float2(o.x, o.y));
          v[2 * q + 1] = add2(v[2 * q + 1], make_float2(o.z, o.w));
        }
      }
    }
    float* to = ws + (size_t)prow * a.Hp + c0 + b0;
#pragma unroll
    for (int q = 0; q < NP / 2; ++q) {
      if constexpr (GB >= 16) {
        if (C::col(4 * q) < lim)
          *reinterpret_cast<float4*>(to + C::col(4 * q)) =
              make_float4(v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * q + i;
          if (C::col(e) < lim) to[C::col(e)] = (e & 1) ? v[e / 2].y : v[e / 2].x;
        }
      }
    }
  };
  partial(acc_pre, a.ws_pre);
  partial(acc, a.ws_post);
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
  if (a.early) pdl_launch_dependents();
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

template <typename D, int GB, bool RUNS, int MAXT, int MINB, int CL>
static cudaError_t run_join_grad_rows(JoinGradArgs& a, const JoinRing& ring, const DeviceInfo& dev, cudaStream_t s) {
  auto kern = join_grad_rows_kernel<D, GB, RUNS, MAXT, MINB, CL>;
  static KernelMemo memo;
  cudaError_t e = memo.allow_smem(kern, dev.max_smem_optin - kJoinStaticSmem, dev);
  if (e != cudaSuccess) return e;
  const int threads = ring.rpc * ring.tpr;
  const int64_t cap = std::min<int64_t>(kJoinMaxPartialsPerSm * dev.sm_count, (a.N + ring.rpc - 1) / ring.rpc);
  FirstLaunch first((unsigned)threads, ring.total, s, CL);
  first.cfg.gridDim = dim3((unsigned)(CL * cap));
  const int resident = memo.resident(threads, ring.total, dev, [&](int* n) {
    if (CL > 1) return cudaOccupancyMaxActiveClusters(n, kern, &first.cfg);
    const cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, threads, ring.total);
    *n *= dev.sm_count;
    return err;
  });
  a.P = (int)std::max<int64_t>(1, std::min<int64_t>(cap, resident));
  a.U = (int)std::min<int64_t>(a.N, (int64_t)a.P * ring.rpc);
  a.early = CL * a.P < dev.sm_count;
  return first.launch((unsigned)(CL * a.P), a.early != 0, kern, a, ring);
}

// CTAs of at most MAXT threads, MINB an SM, in clusters of the fewest CTAs a row
// (CL0 to CL1, powers of two) whose part of it fits the threads and at least two
// row buffers; false where none does.
template <typename D, int GB, bool RUNS, int MAXT, int MINB, int CL0, int CL1>
static bool run_join_grad_shape(JoinGradArgs& a, const DeviceInfo& dev, cudaStream_t s, cudaError_t* e) {
  using C = Chunk<D, GB, kJoinGradCols<D>>;
  const JoinRing r = join_ring<C::E>(a.H, C::ES, C::GE, CL0, RUNS, MAXT, MINB, dev.max_smem_optin);
  if (r.tpr <= MAXT && r.nb >= kJoinMinBuffers) {
    *e = run_join_grad_rows<D, GB, RUNS, MAXT, MINB, CL0>(a, r, dev, s);
    return true;
  }
  if constexpr (CL0 < CL1) return run_join_grad_shape<D, GB, RUNS, MAXT, MINB, 2 * CL0, CL1>(a, dev, s, e);
  return false;
}

// Measured (us, bf16 unless said; in brackets the CTAs a row; groups of narrower
// rows share a CTA):
//   threads x CTAs an SM      160x3      256x2      512x1
//   16384x1280                 63.2       54.0       49.2
//   16384x2048                 70.1       73.9       72.6
//   8192x4096                  76.6 (2)   73.1       71.8
//   8192x5120                  86.8 (2)  102.9 (2)   90.4
//   6000x6144                 103.1 (4)   82.4 (2)   77.0
//   4096x8192                  82.4 (4)   73.6 (2)   71.4
//   4096x10240                 89.7 (4)  111.3 (4)  110.1 (2)
//   2048x16384                 92.8 (8)   78.0 (4)   81.4 (2)
//   8197x2056 fp16, 7 gates    59.5       66.4       55.9
//   fp32 4096x4096             66.8 (4)   70.9 (2)   66.7
//   fp32 2048x8192             70.3 (8)   69.9 (4)   69.2 (2)
// So: one warp a row in 256x2 (its eight groups are a CTA); rows, or groups of
// rows, of up to 512 threads in one CTA; wider ones in clusters, 160x3 where the
// part of at most 256 threads has no more than 160.  fp32, eight columns a thread
// and half the instructions a byte, keeps the large CTA throughout.
//
// Several gate rows: their third parameter vector (join_ring) leaves a CTA that
// is full of threads without its second row buffer: in half precision from 448 to
// 512, 944 to 1024, 1912 to 2048, 3864 to 4096, 7760 to 8192 and 15144 to 16384
// columns.  Those rows go to the clusters of 256x2, of two to eight CTAs of one to
// four warps, with an exchange a row (us, bf16: one gate; eight gate rows; one for
// each 128 rows; in brackets the CTAs a row where they are several):
//   65536x512                  77.4      294.6 (2)  313.3 (2)
//   32768x1024                 74.9      158.8 (2)  181.1 (2)
//   16384x2048                 73.6      111.9 (2)  134.2 (2)
//   16384x2560                 88.4       92.6      118.9
//   8192x4096                  72.9      123.1 (2)  143.6 (2)
//   8192x5120                  87.0 (2)  115.0 (2)  138.2 (2)
//   4096x8192                  71.9      136.3 (4)  141.9 (4)
//   2048x16384                 77.5 (4)  164.2 (8)  166.8 (8)
//   fp32 4096x4096             67.0       71.2
// Past 30272 columns (element by element 30208) nothing fits and the loop runs
// (1024x30720: 81.0 with one gate, 1695 with eight).
template <typename D, int GB, bool RUNS>
static cudaError_t run_join_grad(JoinGradArgs& a, const DeviceInfo& dev, cudaStream_t s, bool* done) {
  cudaError_t e = cudaSuccess;
  *done = true;
  const int whole = chunk_threads(a.H, kJoinGradCols<D>);
  if constexpr (D::VEC == 4) {
    if (whole == 32 && run_join_grad_shape<D, GB, RUNS, 256, 2, 1, 1>(a, dev, s, &e)) return e;
    if (run_join_grad_shape<D, GB, RUNS, 512, 1, 1, 8>(a, dev, s, &e)) return e;
  } else {
    int part = whole;
    while (part > 256) part = (part / 2 + 31) / 32 * 32;
    if (whole > 256 && part <= 160 && run_join_grad_shape<D, GB, RUNS, 160, 3, 2, 8>(a, dev, s, &e)) return e;
    if (whole > 32 && whole <= 512 && run_join_grad_shape<D, GB, RUNS, 512, 1, 1, 1>(a, dev, s, &e)) return e;
    if (run_join_grad_shape<D, GB, RUNS, 256, 2, 1, 8>(a, dev, s, &e)) return e;
  }
  *done = false;
  return cudaSuccess;
}

template <typename D>
cudaError_t launch_join_grad(JoinGradArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  if (a.N == 0) {
    if (a.dgpre == nullptr && a.dgpost == nullptr && a.dgate == nullptr) return cudaSuccess;
    join_grad_zero_kernel<D><<<(unsigned)((a.H + 255) / 256), 256, 0, s>>>(a);
    return cudaGetLastError();
  }
  using T = typename D::T;
  bool done = false;
  cudaError_t e = cudaSuccess;
  if (dev.path != PATH_LOOP) {
    GranuleRule rule;
    rule.add(a.x, a.ldx, sizeof(T));
    if (a.dy) {
      rule.add(a.dy, a.lddy, sizeof(T));
      rule.add(a.h, a.ldh, sizeof(T));
    }
    if (a.dh_in) rule.add(a.dh_in, a.lddh, sizeof(T));
    rule.add(a.dx, a.lddx, sizeof(T));
    rule.add(a.dres, a.lddres, sizeof(T));
    const bool vec = rule.bytes(a.H, sizeof(T)) >= 16, runs = a.gate_rows > 1;
    if (vec)
      e = runs ? run_join_grad<D, 16, true>(a, dev, s, &done) : run_join_grad<D, 16, false>(a, dev, s, &done);
    else
      e = runs ? run_join_grad<D, (int)sizeof(T), true>(a, dev, s, &done)
               : run_join_grad<D, (int)sizeof(T), false>(a, dev, s, &done);
  }
  if (!done) {
    a.P = a.U = (int)std::min<int64_t>(a.N, kJoinMaxPartialsPerSm * dev.sm_count);
    a.early = 0;
    join_grad_loop_kernel<D><<<(unsigned)a.P, kJoinGradLoopThreads, 0, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return launch_join_reduce<D>(a, dev, s);
}

}  // namespace normk
