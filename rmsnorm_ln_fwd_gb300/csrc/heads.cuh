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
// A few flops an element: the traffic bounds both.  16384 tokens of 32+8 heads of
// 128, bf16, run forward in 59 us, 5.7 TB/s in and out; the gradient of 8192 tokens in
// 46 us, 5.5 TB/s.
//
// A head is a group of `lanes` lanes with 16 columns each, chosen so that both
// members of a pair are in one lane: eight columns of each half (or sixteen
// neighbours).  The norm is then a butterfly over the group and the rotation
// needs no exchange.  A warp takes a block of tokens, one a group, and walks their
// heads, the same head of each token at a time: a token's angles are read once, and
// no group idles whatever the number of heads.  (With the groups on one token's heads,
// us, forward and gradient: 16384 tokens of 5+1x128 15.9, 24.8; so 11.1, 20.0.)
#pragma once

#include <algorithm>

#include "chunk.cuh"
#include "common.cuh"
#include "heads.h"

namespace normk {

// Two CTAs (kHeadPerSm) of eight warps an SM.  (us, bf16, 16384 tokens of 32+8x128 and
// 16+16x64 forward: two 59.5, 23.1; three 60.5, 23.0; the gradient at three an SM, 80
// registers, spills.)
constexpr int kHeadWarps = 8;
constexpr int kHeadThreads = 32 * kHeadWarps;

// A lane's 16 columns: [c0, c0 + n0) and [c1, c1 + n1), in halves [0, R/2) and
// [R/2, R), or in halves of the columns past R; with PAIRS neighbours.  CA columns an access.  As fp32,
// pair i (of eight) is element i of `a` and of `b`.
// FULL > 0: heads of FULL columns, all of them rotated, a power of two: what
// follows from that is known at compile time.
template <typename D, int CA, bool PAIRS, int FULL>
struct HeadLane {
  using T = typename D::T;
  static constexpr int ES = (int)sizeof(T);
  static constexpr int NW = 16 * ES / 4;  // packed words
  static constexpr bool kFull = FULL > 0;
  // Halves that no 16 bytes fit (R/2 = 10, 20): copied in the order of the columns, and
  // stored in it by way of shared memory, where a lane's accesses are narrow (32+8 heads
  // of 80 columns, bf16, 20 of them rotated, forward and gradient 162, 198 us with a
  // lane's own accesses to the tensors, 41, 67 so; 112, 56 rotated: 33, 69; 34, 58).
  static constexpr bool STAGED = !PAIRS && ES == 2 && (CA == 4 || CA == 2);
  static constexpr bool ORDERED = PAIRS || STAGED;
  int c0, c1_, n0_, n1_;
  int nr_;  // rotated pairs

  __device__ __forceinline__ int c1() const { return FULL ? c0 + (PAIRS ? 8 : FULL / 2) : c1_; }
  __device__ __forceinline__ int n0() const { return FULL ? 8 : n0_; }
  __device__ __forceinline__ int n1() const { return FULL ? 8 : n1_; }
  __device__ __forceinline__ int nr() const { return FULL ? 8 : nr_; }

  __device__ __forceinline__ HeadLane(int unit, int cols, int R) {
    const int rot = R / 2, units = (rot + 7) / 8;
    if (PAIRS || unit >= units) {
      c0 = PAIRS ? 16 * unit : R + 8 * (unit - units);
      c1_ = c0 + (PAIRS ? 8 : (cols - R + 15) / 16 * 8);
      n0_ = clamp8(min(cols, PAIRS ? cols : R + (cols - R + 15) / 16 * 8) - c0);
      n1_ = clamp8(cols - c1_);
      nr_ = PAIRS ? clamp8(rot - 8 * unit) : 0;
    } else {
      c0 = 8 * unit;
      c1_ = rot + c0;
      n0_ = n1_ = nr_ = clamp8(rot - c0);
    }
  }
  __device__ static __forceinline__ int clamp8(int n) { return n < 0 ? 0 : n > 8 ? 8 : n; }

  // (Half precision by whole accesses is copied to shared memory.)
  __device__ static __forceinline__ void load_half(const T* p, int n, uint32_t* w) {
    static_assert(ES == 4 || CA == 1, "see HeadRing");
    if constexpr (CA * ES == 32) {
      if (n > 0) {
        ld_stream32(p, *reinterpret_cast<uint32_t(*)[8]>(w));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = 0u;
      }
    } else if constexpr (CA * ES == 16) {
#pragma unroll
      for (int k = 0; k < 8 / CA; ++k) {
        const uint4 u = k * CA < n ? ld_stream(p + k * CA) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * k] = u.x;
        w[4 * k + 1] = u.y;
        w[4 * k + 2] = u.z;
        w[4 * k + 3] = u.w;
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
  // PASS: what is stored is the first to leave L2 (16-byte accesses).
  template <bool PASS>
  __device__ static __forceinline__ void store_half(T* p, int n, const uint32_t* w) {
    if constexpr (CA * ES == 32) {
      if (n > 0) st_vec32(p, *reinterpret_cast<const uint32_t(*)[8]>(w));
    } else if constexpr (CA * ES == 16) {
#pragma unroll
      for (int k = 0; k < 8 / CA; ++k) {
        if (k * CA < n) {
          if constexpr (PASS)
            asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p + k * CA), "r"(w[4 * k]), "r"(w[4 * k + 1]),
                         "r"(w[4 * k + 2]), "r"(w[4 * k + 3])
                         : "memory");
          else
            st_vec(p + k * CA, make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
        }
      }
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
    load_half(head + c0, n0(), w);
    load_half(head + c1(), n1(), w + NW / 2);
  }
  // Copy n columns (of eight) into a 16-byte granule of shared memory; zeros for the
  // rest.
  __device__ static __forceinline__ void copy_granule(const T* p, int n, uint32_t to, bool wide) {
    static_assert(ES == 2, "copies of 16 or 8 bytes");
    if (CA == 8 || (STAGED && wide)) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p), "r"(n > 0 ? 16 : 0) : "memory");
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const T* from = 4 * k < n ? p + 4 * k : p;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to + k * 8), "l"(from), "r"(4 * k < n ? 8 : 0) : "memory");
      }
    }
  }
  // Copy the group's part of a head into its lanes' granules: kLaneBytes a lane,
  // the second one of a lane kNext behind the first.  Neighbours are copied in the
  // order of the columns, to addresses in that order, each lane for others: a lane's
  // own two granules in turn, or addresses far apart, ask for each 32-byte sector
  // twice (8192x32+8x128 70.8 us for 49.8).  Halves in the order of the columns gain
  // nothing (128 of which 64 are rotated 24.4 us for 23.8, gradient 41.2 for 38.9).
  static constexpr int kLaneBytes = ORDERED ? 32 : 16, kNext = ORDERED ? 16 : 512;
  __device__ __forceinline__ void copy(const T* head, int unit, int lanes, int cols, uint32_t to, bool wide) const {
    if constexpr (ORDERED) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int g = unit + j * lanes, n = FULL ? 8 : clamp8(cols - 8 * g);
        copy_granule(head + (n ? 8 * g : 0), n, to + (g - 2 * unit) * 16, wide);
      }
    } else {
      copy_granule(head + (n0() ? c0 : 0), n0(), to, wide);
      copy_granule(head + (n1() ? c1() : 0), n1(), to + kNext, wide);
    }
  }
  // The lane's columns from its granules; STAGED: from the group's.
  __device__ __forceinline__ void read(uint32_t from, int unit, uint32_t (&w)[NW]) const {
    if constexpr (!STAGED) {
      lds_words<4>(from, w);
      lds_words<4>(from + kNext, w + 4);
    } else {
      read_half(from - unit * 32 + c0 * 2, n0(), w);
      read_half(from - unit * 32 + c1() * 2, n1(), w + 4);
    }
  }
  __device__ static __forceinline__ void read_half(uint32_t from, int n, uint32_t* w) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = 0u;
#pragma unroll
    for (int k = 0; k < 8 / CA; ++k)
      if (k * CA < n) {
        if constexpr (CA == 2)
          w[k] = lds_u32(from + k * 4);
        else
          lds_words<CA / 2>(from + k * CA * 2, w + k * CA / 2);
      }
  }
  __device__ static __forceinline__ void write_half(uint32_t to, int n, const uint32_t* w) {
#pragma unroll
    for (int k = 0; k < 8 / CA; ++k) {
      if (k * CA < n) {
        if constexpr (CA == 4)
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to + k * 8), "r"(w[2 * k]), "r"(w[2 * k + 1]) : "memory");
        else
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + k * 4), "r"(w[k]) : "memory");
      }
    }
  }
  // Store by way of the lanes' granules at `at`: by all lanes of the warp, `on` those
  // whose group has a head.  The next head's are written behind a barrier (of take).
  __device__ __forceinline__ void store_staged(T* head, bool on, int unit, int lanes, int cols, uint32_t at, bool wide,
                                               const uint32_t (&w)[NW]) const {
    at -= unit * 32;
    write_half(at + c0 * 2, n0(), w);
    write_half(at + c1() * 2, n1(), w + 4);
    __syncwarp();
    if (!on) return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int g = unit + j * lanes, n = clamp8(cols - 8 * g);
      if (n <= 0) continue;
      uint32_t v[4];
      lds_words<4>(at + g * 16, v);
      if (wide) {
        st_vec(head + 8 * g, make_uint4(v[0], v[1], v[2], v[3]));
      } else {
        *reinterpret_cast<uint2*>(head + 8 * g) = make_uint2(v[0], v[1]);
        if (n > 4) *reinterpret_cast<uint2*>(head + 8 * g + 4) = make_uint2(v[2], v[3]);
      }
    }
  }
  template <bool PASS = false>
  __device__ __forceinline__ void store(T* head, const uint32_t (&w)[NW]) const {
    store_half<PASS>(head + c0, n0(), w);
    store_half<PASS>(head + c1(), n1(), w + NW / 2);
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
    if constexpr (PAIRS) return 2 * i < n0() + n1() ? c0 + 2 * i : -1;
    return i < n0() ? c0 + i : -1;
  }
  __device__ __forceinline__ int col_b(int i) const {
    if constexpr (PAIRS) return 2 * i + 1 < n0() + n1() ? c0 + 2 * i + 1 : -1;
    return i < n1() ? c1() + i : -1;
  }
  // Every rotated pair turned by the lane's angles, four granules 512 bytes apart:
  // cos of the first and last four pairs, sin of them (0 past the last rotated pair);
  // the other columns stay, whatever they hold.  BACK: the other way.
  template <bool BACK>
  __device__ __forceinline__ void turn(float2 (&a)[4], float2 (&b)[4], uint32_t angles) const {
    if (PAIRS ? nr() == 8 : nr() > 0) {  // halves have no columns beyond: zeros, and their angles too
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float2 c[2], s[2];
        lds_pairs(angles + 512 * k, c);
        lds_pairs(angles + 1024 + 512 * k, s);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2& x = BACK ? b[2 * k + i] : a[2 * k + i];
          float2& y = BACK ? a[2 * k + i] : b[2 * k + i];
          const float2 u = sub2(mul2(x, c[i]), mul2(y, s[i]));
          y = fma2(y, c[i], mul2(x, s[i]));
          x = u;
        }
      }
    } else if (PAIRS && nr() > 0) {
      float* x = reinterpret_cast<float*>(BACK ? b : a);
      float* y = reinterpret_cast<float*>(BACK ? a : b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i < nr()) {
          const uint32_t at = angles + i / 4 * 512 + i % 4 * 4;
          const float c = __uint_as_float(lds_u32(at)), s = __uint_as_float(lds_u32(at + 1024));
          const float u = x[i] * c - y[i] * s;
          y[i] = fmaf(y[i], c, x[i] * s);
          x[i] = u;
        }
      }
    }
  }
  // The angles of a table row into the lane's granules: copies, where the tables take
  // them (to be waited for), else loads.
  __device__ __forceinline__ void fetch_angles(const HeadArgs& a, int64_t row, int unit, uint32_t to) const {
    if (nr() == 0) return;
    if (a.cvec) {
      const float* c = reinterpret_cast<const float*>(a.cos) + row * a.ldcos + 8 * unit;
      const float* s = reinterpret_cast<const float*>(a.sin) + row * a.ldsin + 8 * unit;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (4 * k < nr()) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to + 512 * k), "l"(c + 4 * k) : "memory");
          asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to + 1024 + 512 * k), "l"(s + 4 * k) : "memory");
        }
      }
    } else {
      const size_t es = a.c_f32 ? 4 : ES;
      const void* c = reinterpret_cast<const unsigned char*>(a.cos) + (row * a.ldcos + 8 * unit) * es;
      const void* s = reinterpret_cast<const unsigned char*>(a.sin) + (row * a.ldsin + 8 * unit) * es;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i < nr()) {
          const uint32_t at = to + i / 4 * 512 + i % 4 * 4;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(load_param<D>(c, i, a.c_f32)) : "memory");
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 1024), "f"(load_param<D>(s, i, a.c_f32)) : "memory");
        }
      }
    }
  }
};

// A lane's parameters in shared memory: 16 floats and four of padding, so that
// the 16-byte reads of eight lanes fall into distinct banks.
constexpr int kHeadSlot = 20;

// gamma of a side in slots (null: ones; 0 past the head).
template <typename Lane, typename D>
__device__ __forceinline__ void head_gamma(float* slots, const HeadArgs& a, const void* g, int t, int nt) {
  for (int unit = t; unit < a.lanes; unit += nt) {
    const Lane l(unit, a.D, a.R);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ca = l.col_a(i), cb = l.col_b(i);
      slots[unit * kHeadSlot + i] = ca < 0 ? 0.f : g ? load_param<D>(g, ca, a.w_f32) : 1.f;
      slots[unit * kHeadSlot + 8 + i] = cb < 0 ? 0.f : g ? load_param<D>(g, cb, a.w_f32) : 1.f;
    }
  }
}

// A token of the batch.
struct HeadToken {
  unsigned b, t;
  __device__ __forceinline__ HeadToken(const HeadArgs& a, unsigned n) : b(a.B == 1 ? 0u : n / (unsigned)a.T), t(n - b * (unsigned)a.T) {}
};

// A warp's share of the work, in units of one head of a block of tokens: the units
// of all blocks, as many as heads each, are shared out evenly, whichever blocks they
// fall into.
struct HeadShare {
  unsigned block;  // of the first one
  int lo, heads;   // which of its units that is
  int64_t left;    // units
  __device__ __forceinline__ HeadShare(const HeadArgs& a, int warp, int heads_) : heads(heads_) {
    const int64_t u = warp * a.each + min((int64_t)warp, a.extra);
    left = a.each + (warp < a.extra);
    block = (unsigned)(u < (int64_t(1) << 31) ? (unsigned)u / (unsigned)heads : u / heads);
    lo = (int)(u - (int64_t)block * heads);
  }
  // Units [from, to) of the block at hand; false behind the last.
  __device__ __forceinline__ bool take(int& from, int& to) {
    if (left <= 0) return false;
    from = lo;
    to = (int)min((int64_t)heads, lo + left);
    left -= to - from;
    lo = 0;
    return true;
  }
};

// Where a token's heads are: I is 32 bits where every tensor of the call has
// fewer than 2^31 elements from its first to its last, else 64.  Offsets of head 0
// of the queries, and of where head 0 would be if the keys' went on behind them.
template <typename I>
struct HeadPlace {
  I q, k;
  __device__ __forceinline__ HeadPlace(const HeadToken& n, const HeadView& vq, const HeadView& vk, int hq)
      : q((I)n.b * (I)vq.sb + (I)n.t * (I)vq.st), k((I)n.b * (I)vk.sb + (I)n.t * (I)vk.st - (I)hq * (I)vk.sh) {}
};
template <typename T, typename I>
__device__ __forceinline__ T* head_at(const HeadView& q, const HeadView& k, const HeadPlace<I>& p, int hq, int h) {
  const bool first = h < hq;
  const I at = first ? p.q + (I)h * (I)q.sh : p.k + (I)h * (I)k.sh;
  return reinterpret_cast<T*>(first ? q.p : k.p) + at;
}

// Heads on their way to a lane: of NT tensors, its columns.  RegisterRing holds one
// head.  CopyRing has copies of SLOTS heads in flight to shared memory (half
// precision, where 16 or 8 bytes can be copied), which no register pays for (gradient,
// 8192x32+8x128 bf16 50.4 -> 45.6 us).  A slot is written again when its values have
// been used, which the head's sums, exchanged by all lanes, tell.
template <typename Lane, typename T, int NT>
struct RegisterRing {
  static constexpr bool COPIES = false;
  static constexpr int SLOTS = 1;
  static constexpr int BYTES = 0;
  uint32_t w[NT][Lane::NW];
  __device__ __forceinline__ RegisterRing(unsigned char*, const HeadArgs&, int, int, int) {}
  __device__ __forceinline__ void fetch(const Lane& me, bool on, const T* (&p)[NT]) {
    if (!on) return;
#pragma unroll
    for (int i = 0; i < NT; ++i) me.load(p[i], w[i]);
  }
  __device__ __forceinline__ void take(const Lane&, uint32_t (&to)[NT][Lane::NW]) const {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < Lane::NW; ++j) to[i][j] = w[i][j];
  }
};
template <typename Lane, typename T, int NT, int SLOTS_>
struct CopyRing {
  static constexpr bool COPIES = true;
  static constexpr int SLOTS = SLOTS_;
  static constexpr int BYTES = SLOTS * NT * 1024;  // of shared memory a warp
  uint32_t base;  // of the lane's granules
  int unit, lanes, cols;
  bool wide;
  int in = 0, out = 0;
  __device__ __forceinline__ CopyRing(unsigned char* smem, const HeadArgs& a, int lane, int unit_, int lanes_)
      : base(smem_u32(smem) + lane * Lane::kLaneBytes), unit(unit_), lanes(lanes_), cols(a.D), wide(a.wide) {}
  // One group of copies a call, with whatever was copied before it; empty without a
  // head.
  __device__ __forceinline__ void fetch(const Lane& me, bool on, const T* (&p)[NT]) {
    if (on) {
#pragma unroll
      for (int i = 0; i < NT; ++i) me.copy(p[i], unit, lanes, cols, base + (in * NT + i) * 1024, wide);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    in = in + 1 == SLOTS ? 0 : in + 1;
  }
  __device__ __forceinline__ void take(const Lane& me, uint32_t (&to)[NT][Lane::NW]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
    __syncwarp();  // every lane's copies are there
#pragma unroll
    for (int i = 0; i < NT; ++i) me.read(base + (out * NT + i) * 1024, unit, to[i]);
    out = out + 1 == SLOTS ? 0 : out + 1;
  }
};
template <typename D, int CA, bool PAIRS, int LANES, int NT>
struct HeadRing {
  using Lane = HeadLane<D, CA, PAIRS, 16 * LANES>;
  using T = typename D::T;
  // Forward (us, 16384 tokens of 32+8x128 and 16+16x64): two slots 59.4, 26.0; three
  // 59.5, 23.1; four 63.4, 22.4.  Backward two fill what shared memory two CTAs leave.
  using Type = std::conditional_t<sizeof(T) == 2 && CA >= 2, CopyRing<Lane, T, NT, NT == 1 ? 3 : 2>, RegisterRing<Lane, T, NT>>;
};

// What runs ahead of a warp's work: the heads into the ring, and, with the first one
// of each block, the angles of its tokens into one of a.bufs sets of the lanes'
// granules.  The position of a group's next token is read a block before.
template <typename D, typename Lane, typename Ring, typename I, int NT>
struct HeadFeed {
  using T = typename D::T;
  static_assert(NT == 1 || NT == 2, "x, or x and dy");
  const HeadArgs& a;
  const Lane& me;
  Ring& ring;
  HeadShare share;
  unsigned token;   // the group's in the block at hand
  int groups, group, unit, hq;
  uint32_t angles;  // the lane's first granule of the first set
  int buf = 0;      // the set to be written next
  unsigned good = 0;  // whether the tokens of each set have positions in the table
  HeadPlace<I> x, dy;
  int h = 0, end = 0;
  bool on = false;
  int64_t pos = 0;  // of the group's token in the next block

  __device__ __forceinline__ HeadFeed(const HeadArgs& a_, const Lane& me_, Ring& ring_, const HeadShare& share_, int groups_,
                                      int group_, int unit_, int hq_, uint32_t angles_)
      : a(a_), me(me_), ring(ring_), share(share_), token(share_.block * groups_ + group_ - groups_), groups(groups_),
        group(group_), unit(unit_), hq(hq_), angles(angles_), x(HeadToken(a_, 0), a_.side[0].x, a_.side[1].x, hq_), dy(x) {
    if constexpr (!Lane::kFull) {  // no angles for pairs that a lane does not have
      for (int i = 0; i < 4 * a.bufs; ++i)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(angles + i * 512), "r"(0u) : "memory");
    }
    if (a.R && share.left > 0) fetch_position(token + groups);
#pragma unroll
    for (int i = 0; i < Ring::SLOTS; ++i) fetch();
  }
  __device__ __forceinline__ void fetch_position(unsigned n) {
    if (n >= a.N) return;
    const HeadToken next(a, n);
    pos = next.t;
    if (a.positions) {
      const int64_t i = next.b * a.pb + next.t * a.pt;
      pos = a.pos64 ? reinterpret_cast<const long long*>(a.positions)[i]
                    : (int64_t) reinterpret_cast<const int*>(a.positions)[i];
    }
  }
  __device__ __forceinline__ void fetch() {
    if (h >= end) {
      if (!share.take(h, end)) {
        h = end = 0;
        on = false;
      } else {
        token += groups;
        on = token < a.N && group < groups;
        if (on) {
          const HeadToken n(a, token);
          x = HeadPlace<I>(n, a.side[0].x, a.side[1].x, hq);
          if (NT > 1) dy = HeadPlace<I>(n, a.side[0].dy, a.side[1].dy, hq);
        }
        if (a.R) {
          const bool fits = pos >= 0 && pos < a.table_rows;
          good = (good & ~(1u << buf)) | ((unsigned)fits << buf);
          if (on && fits) me.fetch_angles(a, pos, unit, angles + buf * 2048);
          if (on && !fits && unit == 0) atomicOr(a.err, kErrBadPosition);
          if constexpr (!Ring::COPIES) asm volatile("cp.async.commit_group;" ::: "memory");
          fetch_position(token + groups);
        } else {
          good = ~0u;
        }
        buf = buf + 1 == a.bufs ? 0 : buf + 1;
      }
    }
    const T* p[NT];
    p[0] = head_at<const T, I>(a.side[0].x, a.side[1].x, x, hq, h);
    if constexpr (NT > 1) p[1] = head_at<const T, I>(a.side[0].dy, a.side[1].dy, dy, hq, h);
    ring.fetch(me, on, p);
    ++h;
  }
};
// At the start of a block's work.
template <typename Ring>
__device__ __forceinline__ void angles_ready() {
  if constexpr (!Ring::COPIES) asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Sum over each `lanes` lanes; LANES: as a compile-time value, or 0.  No power of
// two: a tree into the first one (behind each step, those below `off` hold sums of
// all), which all read.
template <int K, int LANES>
__device__ __forceinline__ void lanes_sum(float (&v)[K], int lanes, int unit) {
  if constexpr (LANES > 0) {
    warp_sum_pow2<K>(v, LANES);
  } else if ((lanes & (lanes - 1)) == 0) {
    warp_sum_pow2<K>(v, lanes);
  } else {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      if (off < lanes) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float other = __shfl_down_sync(0xffffffffu, v[k], off);
          if (unit + off < lanes) v[k] += other;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], (threadIdx.x & 31) - unit);
  }
}

// LANES > 0: heads of 16 * LANES columns, all rotated.
template <typename D, int CA, bool PAIRS, int LANES, typename I>
__global__ void __launch_bounds__(kHeadThreads, kHeadPerSm) head_rotary_kernel(const HeadArgs a) {
  using Lane = HeadLane<D, CA, PAIRS, 16 * LANES>;
  using T = typename D::T;
  using Ring = typename HeadRing<D, CA, PAIRS, LANES, 1>::Type;
  extern __shared__ __align__(16) unsigned char smem[];  // gamma of both sides, each warp's angles and ring
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = LANES ? LANES : a.lanes;
  const int groups = 32 / lanes, group = lane / lanes, unit = lane - group * lanes;
  const Lane me(group < groups ? unit : kHeadMaxCols, a.D, a.R);  // no columns for a lane too many
  const float inv_d = 1.f / (float)a.D;
  const int hq = a.side[0].heads, heads = hq + a.side[1].heads;
  float* slots = reinterpret_cast<float*>(smem);
  unsigned char* at = smem + 2 * lanes * kHeadSlot * 4 + warp * (a.bufs * 2048 + Ring::BYTES + (Lane::STAGED ? 1024 : 0));
  const uint32_t angles = smem_u32(at) + lane * 16;
  pdl_launch_dependents();
  pdl_wait_primary();
  HeadShare work(a, blockIdx.x * kHeadWarps + warp, heads);
  Ring ring(at + a.bufs * 2048, a, lane, unit, lanes);
  const uint32_t stage = smem_u32(at + a.bufs * 2048 + Ring::BYTES) + lane * 32;
  HeadFeed<D, Lane, Ring, I, 1> feed(a, me, ring, work, groups, group, unit, hq, angles);
  for (int k = 0; k < 2; ++k)
    head_gamma<Lane, D>(slots + k * lanes * kHeadSlot, a, a.side[k].gamma, threadIdx.x, kHeadThreads);
  __syncthreads();
  unsigned token = work.block * groups + group;
  int lo, hi, buf = 0;
  for (; work.take(lo, hi); token += groups, buf = buf + 1 == a.bufs ? 0 : buf + 1) {
    const bool on = token < a.N && group < groups;
    const HeadPlace<I> dst(HeadToken(a, on ? token : 0), a.side[0].y, a.side[1].y, hq);
    angles_ready<Ring>();
    const bool good = on && (feed.good >> buf & 1u);
#pragma unroll 1
    for (int h = lo; h < hi; ++h) {
      float2 p[4], q[4];
      {
        uint32_t w[1][Lane::NW];
        ring.take(me, w);
        Lane::unpack(w[0], p, q);
      }
      if constexpr (!Ring::COPIES) feed.fetch();
      float2 sum = splat2(0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = fma2(q[j], q[j], fma2(p[j], p[j], sum));
      float v[1] = {sum.x + sum.y};
      lanes_sum<1, LANES>(v, lanes, unit);
      if constexpr (Ring::COPIES) feed.fetch();
      const float2 r = splat2(rsqrtf(fmaf(v[0], inv_d, a.eps)));
      const uint32_t gamma = smem_u32(slots + ((h < hq ? 0 : lanes) + unit) * kHeadSlot);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 g[2];
        lds_pairs(gamma + 16 * j, g);
        p[2 * j] = mul2(mul2(p[2 * j], r), g[0]);
        p[2 * j + 1] = mul2(mul2(p[2 * j + 1], r), g[1]);
        lds_pairs(gamma + 32 + 16 * j, g);
        q[2 * j] = mul2(mul2(q[2 * j], r), g[0]);
        q[2 * j + 1] = mul2(mul2(q[2 * j + 1], r), g[1]);
      }
      if (!Lane::STAGED && !on) continue;  // no lane exchanges anything below
      uint32_t o[Lane::NW];
      if (good) {
        me.template turn<false>(p, q, angles + buf * 2048);
        Lane::pack(p, q, o);
      } else {  // the token has no position: zeros
#pragma unroll
        for (int j = 0; j < Lane::NW; ++j) o[j] = 0u;
      }
      T* y = head_at<T, I>(a.side[0].y, a.side[1].y, dst, hq, h);
      if constexpr (Lane::STAGED)
        me.store_staged(y, on, unit, lanes, a.D, stage, a.wide, o);
      else if (a.pass)
        me.template store<true>(y, o);
      else
        me.store(y, o);
    }
  }
}

// The gradient.  A lane sums dgamma of its columns, for either side, in granules of
// its own in shared memory (in registers, moved there at a change of sides, fp32
// 4096x32+8x128 47.5 -> 52.3 us); a CTA's sums become its partial row.
template <typename D, int CA, bool PAIRS, int LANES, typename I>
__global__ void __launch_bounds__(kHeadThreads, kHeadPerSm) head_rotary_grad_kernel(const HeadArgs a) {
  using Lane = HeadLane<D, CA, PAIRS, 16 * LANES>;
  using T = typename D::T;
  using Ring = typename HeadRing<D, CA, PAIRS, LANES, 2>::Type;
  extern __shared__ __align__(16) unsigned char smem[];  // gamma of both sides, each warp's sums, then its angles and ring
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = LANES ? LANES : a.lanes;
  const int groups = 32 / lanes, group = lane / lanes, unit = lane - group * lanes;
  const Lane me(group < groups ? unit : kHeadMaxCols, a.D, a.R);  // no columns for a lane too many
  const float inv_d = 1.f / (float)a.D;
  const int hq = a.side[0].heads, heads = hq + a.side[1].heads;
  float* slots = reinterpret_cast<float*>(smem);
  float4* sums = reinterpret_cast<float4*>(slots + 2 * lanes * kHeadSlot);  // [warp][side][granule][lane]
  float4* mine = sums + warp * 256 + lane;
  unsigned char* at = reinterpret_cast<unsigned char*>(sums + kHeadWarps * 256) + warp * (a.bufs * 2048 + Ring::BYTES + (Lane::STAGED ? 1024 : 0));
  const uint32_t angles = smem_u32(at) + lane * 16;
  pdl_launch_dependents();
  pdl_wait_primary();
  HeadShare work(a, blockIdx.x * kHeadWarps + warp, heads);
  Ring ring(at + a.bufs * 2048, a, lane, unit, lanes);
  const uint32_t stage = smem_u32(at + a.bufs * 2048 + Ring::BYTES) + lane * 32;
  HeadFeed<D, Lane, Ring, I, 2> feed(a, me, ring, work, groups, group, unit, hq, angles);
  for (int k = 0; k < 2; ++k)
    head_gamma<Lane, D>(slots + k * lanes * kHeadSlot, a, a.side[k].gamma, threadIdx.x, kHeadThreads);
#pragma unroll
  for (int j = 0; j < 8; ++j) mine[32 * j] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  unsigned token = work.block * groups + group;
  int lo, hi, buf = 0;
  for (; work.take(lo, hi); token += groups, buf = buf + 1 == a.bufs ? 0 : buf + 1) {
    const bool on = token < a.N && group < groups;
    const HeadPlace<I> dst(HeadToken(a, on ? token : 0), a.side[0].y, a.side[1].y, hq);
    angles_ready<Ring>();
    const bool good = on && (feed.good >> buf & 1u);
#pragma unroll 1
    for (int h = lo; h < hi; ++h) {
      float2 p[4], q[4], u[4], v[4];
      {
        uint32_t w[2][Lane::NW];
        ring.take(me, w);
        Lane::unpack(w[0], p, q);
        Lane::unpack(w[1], u, v);
      }
      if constexpr (!Ring::COPIES) feed.fetch();
      const int side = h < hq ? 0 : 1;
      if (good) me.template turn<true>(u, v, angles + buf * 2048);
      float2 sx = splat2(0.f), sw = splat2(0.f);
      const uint32_t gamma = smem_u32(slots + (side * lanes + unit) * kHeadSlot);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 g[2], e[2];
        lds_pairs(gamma + 16 * j, g);
        lds_pairs(gamma + 32 + 16 * j, e);
#pragma unroll
        for (int l = 0; l < 2; ++l) {
          const int c = 2 * j + l;
          sx = fma2(q[c], q[c], fma2(p[c], p[c], sx));
          sw = fma2(mul2(v[c], e[l]), q[c], fma2(mul2(u[c], g[l]), p[c], sw));
        }
      }
      float m[2] = {sx.x + sx.y, sw.x + sw.y};
      lanes_sum<2, LANES>(m, lanes, unit);
      if constexpr (Ring::COPIES) feed.fetch();
      if (!Lane::STAGED && !on) continue;  // no lane exchanges anything below
      uint32_t o[Lane::NW];
      if (good) {
        const float r = rsqrtf(fmaf(m[0], inv_d, a.eps));
        // dx = rstd (w - x rstd^2 mean(w x)); w is formed again rather than kept
        const float2 r2 = splat2(r), k2 = splat2(-(m[1] * inv_d) * r * r);
        float4* sum = mine + side * 128;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 x = sum[32 * j], y = sum[32 * (2 + j)];
          const float2 x0 = fma2(u[2 * j], mul2(p[2 * j], r2), make_float2(x.x, x.y));
          const float2 x1 = fma2(u[2 * j + 1], mul2(p[2 * j + 1], r2), make_float2(x.z, x.w));
          const float2 y0 = fma2(v[2 * j], mul2(q[2 * j], r2), make_float2(y.x, y.y));
          const float2 y1 = fma2(v[2 * j + 1], mul2(q[2 * j + 1], r2), make_float2(y.z, y.w));
          sum[32 * j] = make_float4(x0.x, x0.y, x1.x, x1.y);
          sum[32 * (2 + j)] = make_float4(y0.x, y0.y, y1.x, y1.y);
          float2 g[2], e[2];
          lds_pairs(gamma + 16 * j, g);
          lds_pairs(gamma + 32 + 16 * j, e);
#pragma unroll
          for (int l = 0; l < 2; ++l) {
            const int c = 2 * j + l;
            p[c] = mul2(fma2(p[c], k2, mul2(u[c], g[l])), r2);
            q[c] = mul2(fma2(q[c], k2, mul2(v[c], e[l])), r2);
          }
        }
        Lane::pack(p, q, o);
      } else {  // the token has no position: no gradient
#pragma unroll
        for (int j = 0; j < Lane::NW; ++j) o[j] = 0u;
      }
      T* dx = head_at<T, I>(a.side[0].y, a.side[1].y, dst, hq, h);
      if constexpr (Lane::STAGED)
        me.store_staged(dx, on, unit, lanes, a.D, stage, a.wide, o);
      else
        me.store(dx, o);
    }
  }
  if (!a.want) return;
  __syncthreads();
  // column by column, over groups and warps in a fixed order
  for (int i = threadIdx.x; i < 2 * lanes * 16; i += kHeadThreads) {
    const int k = i / (lanes * 16), l = i / 16 % lanes, e = i % 16;
    float sum = 0.f;
    for (int g = 0; g < groups; ++g) {
      float v[kHeadWarps];  // all in flight: 517 tokens of 9+3x96 8.6 -> 8.1 us
#pragma unroll
      for (int w = 0; w < kHeadWarps; ++w)
        v[w] = reinterpret_cast<const float*>(sums + (w * 2 + k) * 128 + e / 4 * 32 + g * lanes + l)[e % 4];
      sum += tree_sum<kHeadWarps>(v);
    }
    const Lane that(l, a.D, a.R);
    const int col = e < 8 ? that.col_a(e) : that.col_b(e - 8);
    if (col >= 0) a.ws[((int64_t)blockIdx.x * 2 + k) * a.D + col] = sum;
  }
}

// dgamma from the CTAs' partial rows: a CTA takes 32 columns of one side, each
// warp a 32nd of the rows, all of whose loads are in flight at once.
constexpr int kHeadReduceWarps = 32;
template <typename D>
__global__ void __launch_bounds__(32 * kHeadReduceWarps) head_gamma_reduce_kernel(const HeadArgs a, const int rows) {
  __shared__ float sh[kHeadReduceWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane, k = blockIdx.y;
  void* dg = a.side[k].dgamma;
  pdl_launch_dependents();
  pdl_wait_primary();
  const float* ws = a.ws + k * a.D + i;
  float sum = 0.f;
  if (i < a.D) {
    constexpr int B = 10;  // rows a warp has of those of two CTAs an SM
    for (int p = warp; p < rows; p += B * kHeadReduceWarps) {
      float v[B];
#pragma unroll
      for (int j = 0; j < B; ++j)
        v[j] = p + j * kHeadReduceWarps < rows ? ws[(int64_t)(p + j * kHeadReduceWarps) * 2 * a.D] : 0.f;
      sum += tree_sum<B>(v);
    }
  }
  sh[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || i >= a.D || dg == nullptr) return;
  float v[kHeadReduceWarps];
#pragma unroll
  for (int j = 0; j < kHeadReduceWarps; ++j) v[j] = sh[j][lane];
  const float total = tree_sum<kHeadReduceWarps>(v);
  if (a.w_f32)
    reinterpret_cast<float*>(dg)[i] = total;
  else
    store_elem<D>(dg, i, total);
}

// Lanes a head takes: whole units of 16 columns, rounded to a power of two unless
// more heads fit into a warp without.
inline int head_lanes(const HeadArgs& a) {
  const int units = a.interleaved || a.R == 0 ? (a.D + 15) / 16 : (a.R / 2 + 7) / 8 + (a.D - a.R + 15) / 16;
  int lanes = 1;
  while (lanes < units) lanes <<= 1;
  return 32 / units > 32 / lanes ? units : lanes;
}

// Columns an access: eight (16 bytes of half precision, 32 of fp32), four, two (of
// half precision, in halves) or one, whichever divides every column that a lane's
// start at.  Eight and one, and four of fp32 or of neighbours, are the accesses to
// the tensors too, which they have to fit; else a.wide has them 16 or 8 bytes.
template <typename D>
int head_access(HeadArgs& a, bool grad) {
  constexpr int ES = (int)sizeof(typename D::T);
  unsigned long long bits = (unsigned long long)a.D * ES;
  for (const HeadSide& s : a.side) {
    if (!s.heads) continue;
    for (const HeadView* v : {&s.x, &s.y, &s.dy}) {
      if (v == &s.dy && !grad) continue;
      bits |= (unsigned long long)reinterpret_cast<uintptr_t>(v->p);
      bits |= (unsigned long long)((v->sb | v->st | v->sh) * ES);
    }
  }
  const int fit = (bits & (8 * ES - 1)) == 0 ? 8 : (bits & (4 * ES - 1)) == 0 ? 4 : 1;
  a.wide = fit == 8;
  const int half = a.interleaved ? 0 : a.R / 2;
  const int cols = half % 8 == 0 ? 8 : half % 4 == 0 ? 4 : half % 2 == 0 && ES == 2 ? 2 : 1;
  return fit == 1 ? 1 : cols < fit ? cols : fit;
}

// The kernel on as many CTAs as are resident, or fewer.  Its units are shared out
// to the warps one by one: with whole tokens some warps had four and others three of
// 8192 (gradient 56 us for 51.8).  `fixed` bytes of shared memory, `ring` bytes of
// a warp's ring of `slots` heads.
template <typename K>
cudaError_t run_heads(K kern, HeadArgs& a, size_t fixed, int ring, int slots, KernelMemo& memo, const DeviceInfo& dev,
                      cudaStream_t s, int* ctas) {
  const int heads = a.side[0].heads + a.side[1].heads, groups = 32 / a.lanes;
  // sets of angles: of the blocks that a feed of `slots` heads may have entered, and
  // the one at work
  a.bufs = a.R ? (slots + heads - 1) / heads + 1 : 1;
  const size_t smem = fixed + 2 * a.lanes * kHeadSlot * sizeof(float) + (size_t)kHeadWarps * (a.bufs * 2048 + ring);
  if (smem > 48 * 1024) {
    const cudaError_t e = memo.allow_smem(kern, dev.max_smem_optin - 1024, dev);
    if (e != cudaSuccess) return e;
  }
  const int resident = memo.resident(kHeadThreads, smem, dev, [&](int* n) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, kHeadThreads, smem);
    *n = std::min(*n, kHeadPerSm) * dev.sm_count;
    return e;
  });
  const int64_t units = (a.N + groups - 1) / groups * heads;
  *ctas = (int)std::min<int64_t>((units + kHeadWarps - 1) / kHeadWarps, resident);
  a.each = units / ((int64_t)*ctas * kHeadWarps);
  a.extra = units % ((int64_t)*ctas * kHeadWarps);
  const unsigned long long bits = (unsigned long long)reinterpret_cast<uintptr_t>(a.cos) |
                                  (unsigned long long)reinterpret_cast<uintptr_t>(a.sin) |
                                  (unsigned long long)((a.ldcos | a.ldsin) * 4) | (unsigned long long)(a.R / 2 * 4);
  a.cvec = a.c_f32 && (bits & 15) == 0;
  FirstLaunch first(kHeadThreads, smem, s, 1);
  return first.launch((unsigned)*ctas, true, kern, a);
}

template <typename D, int CA, bool PAIRS, int LANES, typename I>
cudaError_t run_head_rotary(HeadArgs a, const DeviceInfo& dev, cudaStream_t s) {
  using Lane = HeadLane<D, CA, PAIRS, 16 * LANES>;
  using Ring = typename HeadRing<D, CA, PAIRS, LANES, 1>::Type;
  // Heads that L2 will not hold until they are read again (a half of its 129 MB, the
  // inputs passing through the other) do not displace the inputs: bf16 32+8x128, 16384
  // tokens 59.8 -> 58.3 us, 16+16x64 25.3 -> 23.9.
  a.pass = a.N * (a.side[0].heads + a.side[1].heads) * a.D * (int64_t)sizeof(typename D::T) > 64000000;
  static KernelMemo memo;
  int ctas;
  return run_heads(head_rotary_kernel<D, CA, PAIRS, LANES, I>, a, 0, Ring::BYTES + Lane::STAGED * 1024, Ring::SLOTS, memo, dev, s,
                   &ctas);
}

template <typename D, int CA, bool PAIRS, int LANES, typename I>
cudaError_t run_head_rotary_grad(HeadArgs a, const DeviceInfo& dev, cudaStream_t s, int* ctas) {
  using Lane = HeadLane<D, CA, PAIRS, 16 * LANES>;
  using Ring = typename HeadRing<D, CA, PAIRS, LANES, 2>::Type;
  static KernelMemo memo;
  return run_heads(head_rotary_grad_kernel<D, CA, PAIRS, LANES, I>, a, kHeadWarps * 4096,
                   Ring::BYTES + Lane::STAGED * 1024, Ring::SLOTS, memo, dev, s, ctas);
}

// Whether every tensor has fewer than 2^31 elements from its first to its last.
inline bool head_offsets_fit(const HeadArgs& a, bool grad) {
  for (const HeadSide& s : a.side) {
    if (!s.heads) continue;
    for (const HeadView* v : {&s.x, &s.y, &s.dy}) {
      if (v == &s.dy && !grad) continue;
      if ((a.B - 1) * v->sb + (a.T - 1) * v->st + (s.heads - 1) * v->sh + a.D >= (int64_t(1) << 31)) return false;
    }
  }
  return true;
}

// f(columns an access, whether pairs are neighbours, lanes a head of 64, 128 or 256
// rotated columns or 0, an offset's type) as compile-time values.
template <typename D, typename F>
cudaError_t head_variants(HeadArgs& a, bool grad, F&& f) {
  const int access = head_access<D>(a, grad);
  auto with = [&](auto ca, auto l, auto off) {
    if constexpr (ca != 2) {
      if (a.interleaved && a.R) return f(ca, std::integral_constant<bool, true>{}, l, off);
    }
    return f(ca, std::integral_constant<bool, false>{}, l, off);
  };
  const std::integral_constant<int, 8> eight;
  const std::integral_constant<int, 4> four;
  const std::integral_constant<int, 2> two;
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 0> any;
  if (!head_offsets_fit(a, grad)) return access == 8 ? with(eight, any, int64_t{}) : with(one, any, int64_t{});
  if (access == 8 && a.R == a.D && a.D == 16 * a.lanes) {
    if (a.D == 64) return with(eight, std::integral_constant<int, 4>{}, uint32_t{});
    if (a.D == 128) return with(eight, std::integral_constant<int, 8>{}, uint32_t{});
    if (a.D == 256) return with(eight, std::integral_constant<int, 16>{}, uint32_t{});
  }
  if constexpr (sizeof(typename D::T) == 2) {
    if (access == 2) return with(two, any, uint32_t{});
  }
  return access == 8 ? with(eight, any, uint32_t{}) : access == 4 ? with(four, any, uint32_t{}) : with(one, any, uint32_t{});
}

template <typename D>
cudaError_t launch_head_rotary(HeadArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  a.err = dev.err;
  a.lanes = head_lanes(a);
  return head_variants<D>(a, false, [&](auto ca, auto pairs, auto l, auto off) {
    return run_head_rotary<D, decltype(ca)::value, decltype(pairs)::value, decltype(l)::value, decltype(off)>(a, dev, s);
  });
}

template <typename D>
cudaError_t launch_head_rotary_grad(HeadArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();
  int rows = 0;
  if (a.N > 0) {
    a.err = dev.err;
    a.lanes = head_lanes(a);
    const cudaError_t e = head_variants<D>(a, true, [&](auto ca, auto pairs, auto l, auto off) {
      return run_head_rotary_grad<D, decltype(ca)::value, decltype(pairs)::value, decltype(l)::value, decltype(off)>(a, dev, s, &rows);
    });
    if (e != cudaSuccess) return e;
  }
  if (!a.want) return cudaSuccess;
  FirstLaunch second(32 * kHeadReduceWarps, 0, s, 1);
  second.cfg.gridDim.y = 2;
  return second.launch((unsigned)((a.D + 31) / 32), true, head_gamma_reduce_kernel<D>, a, rows);
}

}  // namespace normk
