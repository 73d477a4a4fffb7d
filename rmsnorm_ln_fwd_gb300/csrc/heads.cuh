// Per-head RMSNorm with the rotation by position (head_rms_rotary) and its
// gradient.  For head x of a token at position p, with n = x * rstd * gamma,
// rstd = 1/sqrt(mean(x^2) + eps), each pair (a, b) of the first R columns (i and
// i + R/2, or 2i and 2i + 1; c, s the table's column i of row p):
//   y_a = n_a c - n_b s,  y_b = n_b c + n_a s;   y_j = n_j past R.
// Gradient, the rotation being orthogonal up to its scale:
//   u_a = dy_a c + dy_b s,  u_b = dy_b c - dy_a s  (u = dy past R),
//   w = u gamma,  dx = rstd w - x rstd^3 mean(w x),  dgamma = sum of u x rstd.
// The gradient forms rstd again from x, which it reads anyway: a saved one would
// be 4 bytes more a head to write and to read, and both sums of a head meet in
// one exchange.
//
// A few flops an element: the traffic bounds both.
//
// A head is a group of `lanes` lanes with 16 columns each, chosen so that both
// members of a pair are in one lane: eight columns of each half (or sixteen
// neighbours).  The norm is then a butterfly over the group and the rotation
// needs no exchange.  A warp takes a token: its groups walk the token's heads
// with the token's cos and sin in registers, read once a token.
#pragma once

#include <algorithm>

#include "chunk.cuh"
#include "common.cuh"
#include "heads.h"

namespace normk {

constexpr int kHeadWarps = 8;
constexpr int kHeadThreads = 32 * kHeadWarps;

// A lane's 16 columns: [c0, c0 + n0) and [c1, c1 + n1), in halves [0, R/2) and
// [R/2, R), or past R; with PAIRS neighbours.  CA columns an access.  As fp32,
// pair i (of eight) is element i of `a` and of `b`.
template <typename D, int CA, bool PAIRS>
struct HeadLane {
  using T = typename D::T;
  static constexpr int ES = (int)sizeof(T);
  static constexpr int NW = 16 * ES / 4;  // packed words
  int c0, c1, n0, n1;
  int nr;  // rotated pairs
  int p0;  // the first one's table column

  __device__ __forceinline__ HeadLane(int unit, int cols, int R) {
    const int rot = R / 2, units = (rot + 7) / 8;
    if (PAIRS || unit >= units) {
      c0 = PAIRS ? 16 * unit : R + 16 * (unit - units);
      c1 = c0 + 8;
      n0 = clamp8(cols - c0);
      n1 = clamp8(cols - c1);
      p0 = 8 * unit;
      nr = PAIRS ? clamp8(rot - p0) : 0;
    } else {
      c0 = p0 = 8 * unit;
      c1 = rot + c0;
      n0 = n1 = nr = clamp8(rot - c0);
    }
  }
  __device__ static __forceinline__ int clamp8(int n) { return n < 0 ? 0 : n > 8 ? 8 : n; }

  __device__ static __forceinline__ void load_half(const T* p, int n, uint32_t* w) {
    if constexpr (CA * ES == 16) {
#pragma unroll
      for (int k = 0; k < 8 / CA; ++k) {
        const uint4 u = k * CA < n ? ld_stream(p + k * CA) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * k] = u.x;
        w[4 * k + 1] = u.y;
        w[4 * k + 2] = u.z;
        w[4 * k + 3] = u.w;
      }
    } else if constexpr (CA * ES == 8) {
#pragma unroll
      for (int k = 0; k < 8 / CA; ++k) {
        w[2 * k] = w[2 * k + 1] = 0u;
        if (k * CA < n)
          asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[2 * k]), "=r"(w[2 * k + 1]) : "l"(p + k * CA));
      }
    } else if constexpr (ES == 4) {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = k < n ? Chunk<D, ES, 4>::ldg32(p + k) : 0u;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = 2 * k < n ? Chunk<D, ES, 4>::ldg16(p + 2 * k) : 0u;
        const uint32_t hi = 2 * k + 1 < n ? Chunk<D, ES, 4>::ldg16(p + 2 * k + 1) : 0u;
        w[k] = __byte_perm(lo, hi, 0x5410);
      }
    }
  }
  __device__ static __forceinline__ void store_half(T* p, int n, const uint32_t* w) {
    if constexpr (CA * ES == 16) {
#pragma unroll
      for (int k = 0; k < 8 / CA; ++k)
        if (k * CA < n) st_vec(p + k * CA, make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
    } else if constexpr (CA * ES == 8) {
#pragma unroll
      for (int k = 0; k < 8 / CA; ++k)
        if (k * CA < n) *reinterpret_cast<uint2*>(p + k * CA) = make_uint2(w[2 * k], w[2 * k + 1]);
    } else if constexpr (ES == 4) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) reinterpret_cast<uint32_t*>(p)[k] = w[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) reinterpret_cast<uint16_t*>(p)[k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
    }
  }
  __device__ __forceinline__ void load(const T* head, uint32_t (&w)[NW]) const {
    load_half(head + c0, n0, w);
    load_half(head + c1, n1, w + NW / 2);
  }
  __device__ __forceinline__ void store(T* head, const uint32_t (&w)[NW]) const {
    store_half(head + c0, n0, w);
    store_half(head + c1, n1, w + NW / 2);
  }
  __device__ static __forceinline__ void unpack(const uint32_t (&w)[NW], float2 (&a)[4], float2 (&b)[4]) {
    if constexpr (PAIRS) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 u = word_pair<D>(w, 2 * k), v = word_pair<D>(w, 2 * k + 1);
        a[k] = make_float2(u.x, v.x);
        b[k] = make_float2(u.y, v.y);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = word_pair<D>(w, k);
        b[k] = word_pair<D>(w, 4 + k);
      }
    }
  }
  __device__ static __forceinline__ void pack(const float2 (&a)[4], const float2 (&b)[4], uint32_t (&w)[NW]) {
    if constexpr (PAIRS) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        pair_word<D>(w, 2 * k, make_float2(a[k].x, b[k].x));
        pair_word<D>(w, 2 * k + 1, make_float2(a[k].y, b[k].y));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        pair_word<D>(w, k, a[k]);
        pair_word<D>(w, 4 + k, b[k]);
      }
    }
  }
  // Column of pair i's members, or -1 past the head.
  __device__ __forceinline__ int col_a(int i) const {
    if constexpr (PAIRS) return 2 * i < n0 + n1 ? c0 + 2 * i : -1;
    return i < n0 ? c0 + i : -1;
  }
  __device__ __forceinline__ int col_b(int i) const {
    if constexpr (PAIRS) return 2 * i + 1 < n0 + n1 ? c0 + 2 * i + 1 : -1;
    return i < n1 ? c1 + i : -1;
  }
  // gamma of the lane's columns (null: ones), 0 past the head.
  __device__ __forceinline__ void gamma(const void* g, bool f32, float2 (&a)[4], float2 (&b)[4]) const {
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ca = col_a(i), cb = col_b(i);
      v[i] = ca < 0 ? 0.f : g ? load_param<D>(g, ca, f32) : 1.f;
      v[8 + i] = cb < 0 ? 0.f : g ? load_param<D>(g, cb, f32) : 1.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = make_float2(v[2 * k], v[2 * k + 1]);
      b[k] = make_float2(v[8 + 2 * k], v[9 + 2 * k]);
    }
  }
  // The lane's columns of one table row.
  __device__ __forceinline__ void table(const void* t, int64_t row, int64_t ld, bool f32, bool vec, float2 (&c)[4]) const {
    if (vec) {
      const float* p = reinterpret_cast<const float*>(t) + row * ld + p0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 v = 4 * k < nr ? *reinterpret_cast<const float4*>(p + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
        c[2 * k] = make_float2(v.x, v.y);
        c[2 * k + 1] = make_float2(v.z, v.w);
      }
      return;
    }
    const void* p = reinterpret_cast<const unsigned char*>(t) + (row * ld + p0) * (f32 ? 4 : ES);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < nr ? load_param<D>(p, i, f32) : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = make_float2(v[2 * k], v[2 * k + 1]);
  }
  // Every rotated pair turned by (c, s); the others stay, whatever they hold.
  __device__ __forceinline__ void turn(float2 (&a)[4], float2 (&b)[4], const float2 (&c)[4], const float2 (&s)[4]) const {
    if (nr == 8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 m = mul2(b[k], s[k]), u = a[k];
        a[k] = fma2(u, c[k], make_float2(-m.x, -m.y));
        b[k] = fma2(u, s[k], mul2(b[k], c[k]));
      }
    } else if (nr > 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (2 * k < nr) {
          const float u = a[k].x;
          a[k].x = fmaf(u, c[k].x, -(b[k].x * s[k].x));
          b[k].x = fmaf(u, s[k].x, b[k].x * c[k].x);
        }
        if (2 * k + 1 < nr) {
          const float u = a[k].y;
          a[k].y = fmaf(u, c[k].y, -(b[k].y * s[k].y));
          b[k].y = fmaf(u, s[k].y, b[k].y * c[k].y);
        }
      }
    }
  }
};

__device__ __forceinline__ int64_t head_position(const HeadArgs& a, int64_t b, int64_t t) {
  if (a.positions == nullptr) return t;
  const int64_t i = b * a.pb + t * a.pt;
  return a.pos64 ? reinterpret_cast<const long long*>(a.positions)[i] : (int64_t) reinterpret_cast<const int*>(a.positions)[i];
}

// U heads of a group are in flight at a time.
template <typename D, int CA, bool PAIRS, int U>
__global__ void __launch_bounds__(kHeadThreads, 2) head_rotary_kernel(const HeadArgs a) {
  using Lane = HeadLane<D, CA, PAIRS>;
  using T = typename D::T;
  const int lane = threadIdx.x & 31;
  const int groups = 32 / a.lanes, group = lane / a.lanes;
  const Lane me(lane & (a.lanes - 1), a.D, a.R);
  const float inv_d = 1.f / (float)a.D;
  const int heads = a.side[0].heads + a.side[1].heads;
  const int share = ((heads + a.slices - 1) / a.slices + groups - 1) / groups * groups;
  const int64_t items = a.N * a.slices;
  pdl_launch_dependents();
  pdl_wait_primary();
  for (int64_t item = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5); item < items;
       item += (int64_t)gridDim.x * kHeadWarps) {
    const int64_t n = a.slices == 1 ? item : item / a.slices;
    const int slice = a.slices == 1 ? 0 : (int)(item - n * a.slices);
    const int64_t b = a.B == 1 ? 0 : n / a.T, t = n - b * a.T;
    bool good = true;
    float2 c[4], s[4];
    if (a.R) {
      const int64_t pos = head_position(a, b, t);
      good = pos >= 0 && pos < a.table_rows;
      if (good) {
        me.table(a.cos, pos, a.ldcos, a.c_f32, a.cvec, c);
        me.table(a.sin, pos, a.ldsin, a.c_f32, a.cvec, s);
      } else if (lane == 0) {
        atomicOr(a.err, kErrBadPosition);
      }
    }
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const HeadSide& side = a.side[k];
      const int from = max(slice * share - (k ? a.side[0].heads : 0), 0);
      const int to = min((slice + 1) * share - (k ? a.side[0].heads : 0), side.heads);
      if (from >= to) continue;
      float2 ga[4], gb[4];
      me.gamma(side.gamma, a.w_f32, ga, gb);
      const T* x = reinterpret_cast<const T*>(side.x.p) + b * side.x.sb + t * side.x.st;
      T* y = reinterpret_cast<T*>(side.y.p) + b * side.y.sb + t * side.y.st;
#pragma unroll 1
      for (int h = from + group; h - group < to; h += U * groups) {
        uint32_t w[U][Lane::NW];
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (h + i * groups < to) me.load(x + (h + i * groups) * side.x.sh, w[i]);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float2 p[4], q[4];
          Lane::unpack(w[i], p, q);
          float2 sum = splat2(0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) sum = fma2(q[j], q[j], fma2(p[j], p[j], sum));
          float v[1] = {sum.x + sum.y};
          warp_sum_pow2<1>(v, a.lanes);
          const float2 r = splat2(good ? rsqrtf(fmaf(v[0], inv_d, a.eps)) : 0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = mul2(mul2(p[j], r), ga[j]);
            q[j] = mul2(mul2(q[j], r), gb[j]);
          }
          me.turn(p, q, c, s);
          Lane::pack(p, q, w[i]);
          if (!good) {
#pragma unroll
            for (int j = 0; j < Lane::NW; ++j) w[i][j] = 0u;
          }
          if (h + i * groups < to) me.store(y + (h + i * groups) * side.y.sh, w[i]);
        }
      }
    }
  }
}

// The gradient.  A CTA takes one side (queries: the first a.ctas[0] CTAs), whose
// warps walk the tokens with each column's part of dgamma in registers; the parts
// meet in shared memory and become the CTA's partial row.
template <typename D, int CA, bool PAIRS, int U>
__global__ void __launch_bounds__(kHeadThreads, 2) head_rotary_grad_kernel(const HeadArgs a) {
  using Lane = HeadLane<D, CA, PAIRS>;
  using T = typename D::T;
  extern __shared__ float parts[];  // [warps][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = 32 / a.lanes, group = lane / a.lanes;
  const Lane me(lane & (a.lanes - 1), a.D, a.R);
  const float inv_d = 1.f / (float)a.D;
  const bool keys = (int)blockIdx.x >= a.ctas[0];
  const HeadSide& side = a.side[keys];
  const int cta = keys ? blockIdx.x - a.ctas[0] : blockIdx.x, ctas = a.ctas[keys], slices = a.slice[keys];
  const int share = ((side.heads + slices - 1) / slices + groups - 1) / groups * groups;
  const int64_t items = a.N * slices;
  float2 da[4], db[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) da[j] = db[j] = splat2(0.f);
  pdl_launch_dependents();
  pdl_wait_primary();
  float2 ga[4], gb[4];
  me.gamma(side.gamma, a.w_f32, ga, gb);
  for (int64_t item = (int64_t)cta * kHeadWarps + warp; item < items; item += (int64_t)ctas * kHeadWarps) {
    const int64_t n = slices == 1 ? item : item / slices;
    const int from = slices == 1 ? 0 : (int)(item - n * slices) * share, to = min(from + share, side.heads);
    const int64_t b = a.B == 1 ? 0 : n / a.T, t = n - b * a.T;
    bool good = true;
    float2 c[4], s[4];
    if (a.R) {
      const int64_t pos = head_position(a, b, t);
      good = pos >= 0 && pos < a.table_rows;
      if (good) {
        me.table(a.cos, pos, a.ldcos, a.c_f32, a.cvec, c);
        me.table(a.sin, pos, a.ldsin, a.c_f32, a.cvec, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = make_float2(-s[j].x, -s[j].y);
      } else if (lane == 0) {
        atomicOr(a.err, kErrBadPosition);
      }
    }
    const T* x = reinterpret_cast<const T*>(side.x.p) + b * side.x.sb + t * side.x.st;
    const T* dy = reinterpret_cast<const T*>(side.dy.p) + b * side.dy.sb + t * side.dy.st;
    T* dx = reinterpret_cast<T*>(side.y.p) + b * side.y.sb + t * side.y.st;
#pragma unroll 1
    for (int h = from + group; h - group < to; h += U * groups) {
      uint32_t w[U][Lane::NW], g[U][Lane::NW];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (h + i * groups < to) {
          me.load(x + (h + i * groups) * side.x.sh, w[i]);
          me.load(dy + (h + i * groups) * side.dy.sh, g[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float2 p[4], q[4], u[4], v[4];
        Lane::unpack(w[i], p, q);
        Lane::unpack(g[i], u, v);
        me.turn(u, v, c, s);
        float2 sx = splat2(0.f), sw = splat2(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sx = fma2(q[j], q[j], fma2(p[j], p[j], sx));
          sw = fma2(mul2(v[j], gb[j]), q[j], fma2(mul2(u[j], ga[j]), p[j], sw));
        }
        float m[2] = {sx.x + sx.y, sw.x + sw.y};
        warp_sum_pow2<2>(m, a.lanes);
        const float r = rsqrtf(fmaf(m[0], inv_d, a.eps));
        // dx = rstd (w - x rstd^2 mean(w x))
        const float2 r2 = splat2(r), k2 = splat2(-(m[1] * inv_d) * r * r);
        if (good && h + i * groups < to) {
          float2 o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            da[j] = fma2(u[j], mul2(p[j], r2), da[j]);
            db[j] = fma2(v[j], mul2(q[j], r2), db[j]);
            o[j] = mul2(fma2(p[j], k2, mul2(u[j], ga[j])), r2);
            q[j] = mul2(fma2(q[j], k2, mul2(v[j], gb[j])), r2);
          }
          Lane::pack(o, q, w[i]);
        }
        if (!good) {
#pragma unroll
          for (int j = 0; j < Lane::NW; ++j) w[i][j] = 0u;
        }
        if (h + i * groups < to) me.store(dx + (h + i * groups) * side.y.sh, w[i]);
      }
    }
  }
  if (!a.want) return;
  // groups of a warp, then the warps, in a fixed order
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[4] = {da[j].x, da[j].y, db[j].x, db[j].y};
    for (int off = a.lanes; off < 32; off <<= 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    }
    if (group == 0) {
      float* row = parts + warp * a.D;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (me.col_a(2 * j + i) >= 0) row[me.col_a(2 * j + i)] = v[i];
        if (me.col_b(2 * j + i) >= 0) row[me.col_b(2 * j + i)] = v[2 + i];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.D; i += kHeadThreads) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kHeadWarps; ++w) sum += parts[w * a.D + i];
    a.ws[(int64_t)blockIdx.x * a.D + i] = sum;
  }
}

// dgamma from its side's partial rows: a CTA takes 32 columns of one side, its
// warps rows in turn.
template <typename D>
__global__ void __launch_bounds__(512) head_gamma_reduce_kernel(const HeadArgs a) {
  __shared__ float sh[16][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane, k = blockIdx.y;
  void* dg = a.side[k].dgamma;
  pdl_launch_dependents();
  pdl_wait_primary();
  const float* ws = a.ws + (int64_t)(k ? a.ctas[0] : 0) * a.D + i;
  float sum = 0.f;
  if (i < a.D) {
#pragma unroll 4
    for (int p = warp; p < a.ctas[k]; p += 16) sum += ws[(int64_t)p * a.D];
  }
  sh[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || i >= a.D || dg == nullptr) return;
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = sh[j][lane];
  const float total = tree_sum<16>(v);
  if (a.w_f32)
    reinterpret_cast<float*>(dg)[i] = total;
  else
    store_elem<D>(dg, i, total);
}

// Lanes a head takes: whole units of 16 columns, rounded to a power of two.
inline int head_lanes(const HeadArgs& a) {
  const int units = a.interleaved || a.R == 0 ? (a.D + 15) / 16 : (a.R / 2 + 7) / 8 + (a.D - a.R + 15) / 16;
  int lanes = 1;
  while (lanes < units) lanes <<= 1;
  return lanes;
}

// Columns an access: 16 bytes, 8, or one element, whichever divides every
// column that an access starts at, and fits every tensor.
template <typename D>
int head_access(const HeadArgs& a, bool grad) {
  constexpr int ES = (int)sizeof(typename D::T);
  unsigned long long bits = (unsigned long long)a.D * ES;
  bits |= (unsigned long long)(a.interleaved || a.R == 0 ? 0 : a.R / 2) * ES;
  for (const HeadSide& s : a.side) {
    if (!s.heads) continue;
    for (const HeadView* v : {&s.x, &s.y, &s.dy}) {
      if (v == &s.dy && !grad) continue;
      bits |= (unsigned long long)reinterpret_cast<uintptr_t>(v->p);
      bits |= (unsigned long long)((v->sb | v->st | v->sh) * ES);
    }
  }
  return (bits & 15) == 0 ? 16 / ES : ES == 2 && (bits & 7) == 0 ? 4 : 1;
}

template <typename D>
void head_plan(HeadArgs& a, const DeviceInfo& dev) {
  a.err = dev.err;
  a.lanes = head_lanes(a);
  const unsigned long long bits = (unsigned long long)reinterpret_cast<uintptr_t>(a.cos) |
                                  (unsigned long long)reinterpret_cast<uintptr_t>(a.sin) |
                                  (unsigned long long)((a.ldcos | a.ldsin) * 4) | (unsigned long long)(a.R / 2 * 4);
  a.cvec = a.R && a.c_f32 && (bits & 15) == 0;
}

// Warps that share a token's heads: more than one where tokens are few.
inline int head_slices(const HeadArgs& a, int heads, int64_t warps) {
  const int groups = 32 / a.lanes;
  const int64_t most = (heads + groups - 1) / groups, want = (warps + a.N - 1) / a.N;
  return (int)std::max<int64_t>(1, std::min(most, want));
}

template <typename D, int CA, bool PAIRS>
cudaError_t run_head_rotary(HeadArgs a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int U = sizeof(typename D::T) == 2 ? 4 : 2;
  a.slices = head_slices(a, a.side[0].heads + a.side[1].heads, (int64_t)dev.sm_count * 16);
  const int64_t ctas = (a.N * a.slices + kHeadWarps - 1) / kHeadWarps;
  FirstLaunch first(kHeadThreads, 0, s, 1);
  return first.launch((unsigned)std::min<int64_t>(ctas, 1 << 20), true, head_rotary_kernel<D, CA, PAIRS, U>, a);
}

template <typename D, int CA, bool PAIRS>
cudaError_t run_head_rotary_grad(HeadArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int U = sizeof(typename D::T) == 2 ? 2 : 1;
  auto kern = head_rotary_grad_kernel<D, CA, PAIRS, U>;
  const size_t smem = a.want ? sizeof(float) * kHeadWarps * a.D : 0;
  static KernelMemo memo;
  const int resident = memo.resident(kHeadThreads, smem, dev, [&](int* n) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, kHeadThreads, smem);
    *n = std::min(*n, kHeadGradMaxPerSm) * dev.sm_count;
    return e;
  });
  // the resident CTAs, shared by the sides as their heads are
  const int heads = a.side[0].heads + a.side[1].heads;
  for (int k = 0; k < 2; ++k) {
    a.ctas[k] = 0;
    if (!a.side[k].heads) continue;
    const int most = std::max(1, (int)((int64_t)resident * a.side[k].heads / heads));
    a.slice[k] = head_slices(a, a.side[k].heads, (int64_t)most * kHeadWarps);
    a.ctas[k] = (int)std::min<int64_t>((a.N * a.slice[k] + kHeadWarps - 1) / kHeadWarps, most);
  }
  FirstLaunch first(kHeadThreads, smem, s, 1);
  return first.launch((unsigned)(a.ctas[0] + a.ctas[1]), true, kern, a);
}

// f(columns an access, whether pairs are neighbours) as compile-time values.
template <typename D, typename F>
cudaError_t head_variants(int access, bool pairs, F&& f) {
  constexpr int V = 16 / (int)sizeof(typename D::T);
  auto with = [&](auto ca) {
    return pairs ? f(ca, std::integral_constant<bool, true>{}) : f(ca, std::integral_constant<bool, false>{});
  };
  if (access == V) return with(std::integral_constant<int, V>{});
  if constexpr (V == 8) {
    if (access == 4) return with(std::integral_constant<int, 4>{});
  }
  return with(std::integral_constant<int, 1>{});
}

template <typename D>
cudaError_t launch_head_rotary(HeadArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  head_plan<D>(a, dev);
  return head_variants<D>(head_access<D>(a, false), a.interleaved && a.R, [&](auto ca, auto pairs) {
    return run_head_rotary<D, decltype(ca)::value, decltype(pairs)::value>(a, dev, s);
  });
}

template <typename D>
cudaError_t launch_head_rotary_grad(HeadArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();
  a.ctas[0] = a.ctas[1] = 0;
  if (a.N > 0) {
    head_plan<D>(a, dev);
    const cudaError_t e = head_variants<D>(head_access<D>(a, true), a.interleaved && a.R, [&](auto ca, auto pairs) {
      return run_head_rotary_grad<D, decltype(ca)::value, decltype(pairs)::value>(a, dev, s);
    });
    if (e != cudaSuccess) return e;
  }
  if (!a.want) return cudaSuccess;
  FirstLaunch second(512, 0, s, 1);
  second.cfg.gridDim.y = 2;
  return second.launch((unsigned)((a.D + 31) / 32), true, head_gamma_reduce_kernel<D>, a);
}

}  // namespace normk
