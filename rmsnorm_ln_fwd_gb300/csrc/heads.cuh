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
// 128, bf16, run forward in 60 us, 5.6 TB/s in and out, and stores without the
// arithmetic in 59; the gradient of 8192 tokens in 46 us, 5.5 TB/s.
//
// A head is a group of `lanes` lanes with 16 columns each, chosen so that both
// members of a pair are in one lane: eight columns of each half (or sixteen
// neighbours).  The norm is then a butterfly over the group and the rotation
// needs no exchange.  A warp takes a token, or a part of its heads: its groups walk
// them with the token's cos and sin in shared memory, read once a token.
#pragma once

#include <algorithm>

#include "chunk.cuh"
#include "common.cuh"
#include "heads.h"

namespace normk {

// Two CTAs (kHeadPerSm) of eight warps an SM, up to 128 registers.  (us, 16384 tokens of 32+8
// heads of 128 bf16 forward, and 8192 backward while the gradient still held its next
// head in registers: 59.8, 51.8; five CTAs of four warps 59.9, 57; three of six 59.4,
// 68; three of eight, 80 registers, 59.8, 69.)
constexpr int kHeadWarps = 8;
constexpr int kHeadThreads = 32 * kHeadWarps;

// A lane's 16 columns: [c0, c0 + n0) and [c1, c1 + n1), in halves [0, R/2) and
// [R/2, R), or past R; with PAIRS neighbours.  CA columns an access.  As fp32,
// pair i (of eight) is element i of `a` and of `b`.
// FULL > 0: heads of FULL columns, all of them rotated, a power of two: what
// follows from that is known at compile time.
template <typename D, int CA, bool PAIRS, int FULL>
struct HeadLane {
  using T = typename D::T;
  static constexpr int ES = (int)sizeof(T);
  static constexpr int NW = 16 * ES / 4;  // packed words
  int c0, c1_, n0_, n1_;
  int nr_;  // rotated pairs

  __device__ __forceinline__ int c1() const { return FULL ? c0 + (PAIRS ? 8 : FULL / 2) : c1_; }
  __device__ __forceinline__ int n0() const { return FULL ? 8 : n0_; }
  __device__ __forceinline__ int n1() const { return FULL ? 8 : n1_; }
  __device__ __forceinline__ int nr() const { return FULL ? 8 : nr_; }

  __device__ __forceinline__ HeadLane(int unit, int cols, int R) {
    const int rot = R / 2, units = (rot + 7) / 8;
    if (PAIRS || unit >= units) {
      c0 = PAIRS ? 16 * unit : R + 16 * (unit - units);
      c1_ = c0 + 8;
      n0_ = clamp8(cols - c0);
      n1_ = clamp8(cols - c1_);
      nr_ = PAIRS ? clamp8(rot - 8 * unit) : 0;
    } else {
      c0 = 8 * unit;
      c1_ = rot + c0;
      n0_ = n1_ = nr_ = clamp8(rot - c0);
    }
  }
  __device__ static __forceinline__ int clamp8(int n) { return n < 0 ? 0 : n > 8 ? 8 : n; }

  __device__ static __forceinline__ void load_half(const T* p, int n, uint32_t* w) {
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
  __device__ static __forceinline__ void copy_granule(const T* p, int n, uint32_t to) {
    constexpr int B = CA * ES;
    static_assert(ES == 2 && (B == 16 || B == 8), "copies of 16 or 8 bytes");
#pragma unroll
    for (int k = 0; k < 8 / CA; ++k) {
      const T* from = k * CA < n ? p + k * CA : p;
      if constexpr (B == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(k * CA < n ? 16 : 0) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to + k * B), "l"(from), "r"(k * CA < n ? 8 : 0) : "memory");
    }
  }
  // Copy the group's part of a head into its lanes' granules: kLaneBytes a lane,
  // the second one of a lane kNext behind the first.  Neighbours are copied in the
  // order of the columns, to addresses in that order, each lane for others: a lane's
  // own two granules in turn, or addresses far apart, ask for each 32-byte sector
  // twice (8192x32+8x128 70.8 us for 49.8).
  static constexpr int kLaneBytes = PAIRS ? 32 : 16, kNext = PAIRS ? 16 : 512;
  __device__ __forceinline__ void copy(const T* head, int unit, int lanes, int cols, uint32_t to) const {
    if constexpr (PAIRS) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int g = unit + j * lanes, n = FULL ? 8 : clamp8(cols - 8 * g);
        copy_granule(head + (n ? 8 * g : 0), n, to + (g - 2 * unit) * 16);
      }
    } else {
      copy_granule(head + (n0() ? c0 : 0), n0(), to);
      copy_granule(head + (n1() ? c1() : 0), n1(), to + kNext);
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
  // Every rotated pair turned by the angles in the lane's slot; the others stay,
  // whatever they hold.  BACK: the other way.
  template <bool BACK>
  __device__ __forceinline__ void turn(float2 (&a)[4], float2 (&b)[4], uint32_t slot) const {
    if (nr() == 8) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float2 c[2], s[2];
        lds_pairs(slot + 16 * k, c);
        lds_pairs(slot + 32 + 16 * k, s);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2& x = BACK ? b[2 * k + i] : a[2 * k + i];
          float2& y = BACK ? a[2 * k + i] : b[2 * k + i];
          const float2 u = sub2(mul2(x, c[i]), mul2(y, s[i]));
          y = fma2(y, c[i], mul2(x, s[i]));
          x = u;
        }
      }
    } else if (nr() > 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float* x = reinterpret_cast<float*>(BACK ? b : a);
        float* y = reinterpret_cast<float*>(BACK ? a : b);
#pragma unroll
        for (int i = 2 * k; i < 2 * k + 2; ++i) {
          if (i < nr()) {
            const float c = __uint_as_float(lds_u32(slot + 4 * i)), s = __uint_as_float(lds_u32(slot + 32 + 4 * i));
            const float u = x[i] * c - y[i] * s;
            y[i] = fmaf(y[i], c, x[i] * s);
            x[i] = u;
          }
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
  __device__ __forceinline__ void step(const HeadArgs& a) {
    if (++t == (unsigned)a.T) {
      t = 0;
      ++b;
    }
  }
};

// A warp's share of the work, in units of one head a group: the units of all
// tokens, a.its each, are shared out evenly, whichever tokens they fall into.
struct HeadShare {
  unsigned first;  // the token of the first one
  int lo;          // and which of its units that is
  int64_t left;    // units
  __device__ __forceinline__ HeadShare(const HeadArgs& a, int warp) {
    const int64_t u = warp * a.each + min((int64_t)warp, a.extra);
    left = a.each + (warp < a.extra);
    first = (unsigned)(u < (int64_t(1) << 31) ? (unsigned)u / (unsigned)a.its : u / a.its);
    lo = (int)(u - (int64_t)first * a.its);
  }
  // Units [lo, hi) of the token at hand; false behind the last.
  __device__ __forceinline__ bool take(const HeadArgs& a, int& from, int& to) {
    if (left <= 0) return false;
    from = lo;
    to = (int)min((int64_t)a.its, lo + left);
    left -= to - from;
    lo = 0;
    return true;
  }
};

// The angles of a warp's tokens: positions two tokens ahead and table rows one
// ahead are in registers, the token's own angles in the warp's slots.
template <typename D, int LANES>
struct HeadAngles {
  static constexpr int AHEAD = LANES == 16 ? 8 : 4;  // values of a table row a lane holds: 128 or 256
  const HeadArgs& a;
  float* slots;
  int lane;
  HeadToken ahead;  // the token whose position is to be fetched
  int tokens;       // that are left from it on
  int64_t pos;      // the position of the token after the next one
  int64_t row;      // the next one's, and its table row
  float v[AHEAD];
  bool next_good;

  __device__ __forceinline__ HeadAngles(const HeadArgs& a_, float* slots_, int lane_, const HeadToken& first, int tokens_)
      : a(a_), slots(slots_), lane(lane_), ahead(first), tokens(tokens_), pos(0), row(0), next_good(true) {
    if (!a.R) return;
    fetch_position();
    fetch_row();
    fetch_position();
  }
  __device__ __forceinline__ void fetch_position() {
    if (tokens-- <= 0) return;
    pos = ahead.t;
    if (a.positions) {
      const int64_t i = ahead.b * a.pb + ahead.t * a.pt;
      pos = a.pos64 ? reinterpret_cast<const long long*>(a.positions)[i]
                    : (int64_t) reinterpret_cast<const int*>(a.positions)[i];
    }
    ahead.step(a);
  }
  // Value e of the row [cos | sin].
  __device__ __forceinline__ float value(int e) const {
    const int half = a.R / 2;
    const void* t = e < half ? a.cos : a.sin;
    const int64_t at = row * (e < half ? a.ldcos : a.ldsin) + (e < half ? e : e - half);
    return a.c_f32 ? reinterpret_cast<const float*>(t)[at] : load_elem<D>(t, at);
  }
  __device__ __forceinline__ void put(int e, float x) const {
    const int half = a.R / 2, i = e < half ? e : e - half;
    slots[i / 8 * kHeadSlot + i % 8 + (e < half ? 0 : 8)] = x;
  }
  __device__ __forceinline__ void fetch_row() {
    row = pos;
    next_good = row >= 0 && row < a.table_rows;
    if (!next_good) return;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (lane + 32 * k < a.R) v[k] = value(lane + 32 * k);
  }
  // The next token's angles go into the slots, and those after it are asked for.
  // Whether its position is in the table.
  __device__ __forceinline__ bool turn_over() {
    if (!a.R) return true;
    const bool good = next_good;
    __syncwarp();  // the lanes are through with the angles before
    if (good) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (lane + 32 * k < a.R) put(lane + 32 * k, v[k]);
      for (int e = lane + 32 * AHEAD; e < a.R; e += 32) put(e, value(e));
    } else if (lane == 0) {
      atomicOr(a.err, kErrBadPosition);
    }
    __syncwarp();
    fetch_row();
    fetch_position();
    return good;
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

// The gradient's inputs on their way to a lane: x and dy of its columns.
// RegisterRing holds one head.  CopyRing has copies of two in flight to shared
// memory (half precision, where 16 or 8 bytes can be copied), which no register
// pays for: bf16 8192x32+8x128 50.4 -> 45.6 us.  A slot is written again an
// iteration after its values were used, with the head's sums, which all lanes
// exchange, in between.
template <typename Lane, typename T>
struct RegisterRing {
  static constexpr int AHEAD = 1;
  static constexpr int BYTES = 0;  // of shared memory a warp
  uint32_t x[Lane::NW], y[Lane::NW];
  __device__ __forceinline__ RegisterRing(unsigned char*, int, int, int, int) {}
  __device__ __forceinline__ void fetch(const Lane& me, bool on, const T* px, const T* py) {
    if (!on) return;
    me.load(px, x);
    me.load(py, y);
  }
  __device__ __forceinline__ void take(uint32_t (&tx)[Lane::NW], uint32_t (&ty)[Lane::NW]) const {
#pragma unroll
    for (int j = 0; j < Lane::NW; ++j) {
      tx[j] = x[j];
      ty[j] = y[j];
    }
  }
};
template <typename Lane, typename T>
struct CopyRing {
  static constexpr int AHEAD = 2;
  static constexpr int SLOTS = AHEAD + 1;
  static constexpr int BYTES = SLOTS * 2048;
  uint32_t base;  // of the lane's granules
  int unit, lanes, cols;
  int in = 0, out = 0;
  __device__ __forceinline__ CopyRing(unsigned char* smem, int lane, int unit_, int lanes_, int cols_)
      : base(smem_u32(smem) + lane * Lane::kLaneBytes), unit(unit_), lanes(lanes_), cols(cols_) {}
  // One group of copies a call, empty without a head.
  __device__ __forceinline__ void fetch(const Lane& me, bool on, const T* px, const T* py) {
    if (on) {
      me.copy(px, unit, lanes, cols, base + in * 2048);
      me.copy(py, unit, lanes, cols, base + in * 2048 + 1024);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    in = in + 1 == SLOTS ? 0 : in + 1;
  }
  __device__ __forceinline__ void take(uint32_t (&tx)[Lane::NW], uint32_t (&ty)[Lane::NW]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
    __syncwarp();  // every lane's copies are there
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      lds_words<4>(base + out * 2048 + j * Lane::kNext, tx + 4 * j);
      lds_words<4>(base + out * 2048 + 1024 + j * Lane::kNext, ty + 4 * j);
    }
    out = out + 1 == SLOTS ? 0 : out + 1;
  }
};

// Sum over each `lanes` lanes; LANES: as a compile-time value, or 0.
template <int K, int LANES>
__device__ __forceinline__ void lanes_sum(float (&v)[K], int lanes) {
  warp_sum_pow2<K>(v, LANES ? LANES : lanes);
}

// U heads of a group are in flight, over the ends of tokens, while as many are at
// work.  LANES > 0: heads of 16 * LANES columns, all rotated.
template <typename D, int CA, bool PAIRS, int U, int LANES, typename I>
__global__ void __launch_bounds__(kHeadThreads, kHeadPerSm) head_rotary_kernel(const HeadArgs a) {
  using Lane = HeadLane<D, CA, PAIRS, 16 * LANES>;
  using T = typename D::T;
  extern __shared__ __align__(16) float slots[];  // gamma of both sides, each warp's angles
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = LANES ? LANES : a.lanes;
  const int groups = 32 / lanes, group = lane / lanes, unit = lane & (lanes - 1);
  const Lane me(unit, a.D, a.R);
  const float inv_d = 1.f / (float)a.D;
  const int hq = a.side[0].heads, heads = hq + a.side[1].heads;
  const uint32_t gammas = smem_u32(slots + unit * kHeadSlot);
  float* angles = slots + (2 + warp) * lanes * kHeadSlot;
  const uint32_t angle = smem_u32(angles + unit * kHeadSlot);
  pdl_launch_dependents();
  pdl_wait_primary();
  HeadShare share(a, blockIdx.x * kHeadWarps + warp);
  HeadToken token(a, share.first);
  const int tokens = share.left > 0 ? (int)((share.lo + share.left + a.its - 1) / a.its) : 0;
  HeadPlace<I> src(token, a.side[0].x, a.side[1].x, hq), dst(token, a.side[0].y, a.side[1].y, hq);
  uint32_t next[U][Lane::NW];
  auto fetch = [&](int h, int to) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (h + i * groups < to) me.load(head_at<T, I>(a.side[0].x, a.side[1].x, src, hq, h + i * groups), next[i]);
  };
  int lo, hi, from, to;
  // the next token's units as heads [from, to), whose first ones are asked for
  auto enter = [&] {
    if (!share.take(a, lo, hi)) return false;
    from = lo * groups + group;
    to = min(hi * groups, heads);
    src = HeadPlace<I>(token, a.side[0].x, a.side[1].x, hq);
    dst = HeadPlace<I>(token, a.side[0].y, a.side[1].y, hq);
    token.step(a);
    fetch(from, to);
    return true;
  };
  HeadAngles<D, LANES> way(a, angles, lane, token, tokens);
  bool on = enter();
  for (int k = 0; k < 2; ++k)
    head_gamma<Lane, D>(slots + k * lanes * kHeadSlot, a, a.side[k].gamma, threadIdx.x, kHeadThreads);
  __syncthreads();
  while (on) {
    const bool good = way.turn_over();
    const HeadPlace<I> here = dst;
    const int end = to;
#pragma unroll 1
    for (int h = from, more = 1; more; h += U * groups) {
      uint32_t now[U][Lane::NW];
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < Lane::NW; ++j) now[i][j] = next[i][j];
      more = h - group + U * groups < end;
      if (more)
        fetch(h + U * groups, end);
      else
        on = enter();
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int k = h + i * groups;
        if (k - group >= end) break;  // the same for the whole warp
        float2 p[4], q[4];
        Lane::unpack(now[i], p, q);
        float2 sum = splat2(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = fma2(q[j], q[j], fma2(p[j], p[j], sum));
        float v[1] = {sum.x + sum.y};
        lanes_sum<1, LANES>(v, lanes);
        const float2 r = splat2(rsqrtf(fmaf(v[0], inv_d, a.eps)));
        const uint32_t gamma = gammas + (k < hq ? 0 : lanes * kHeadSlot * 4);
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
        if (good) {
          me.template turn<false>(p, q, angle);
          Lane::pack(p, q, now[i]);
        } else {  // the token has no position: zeros
#pragma unroll
          for (int j = 0; j < Lane::NW; ++j) now[i][j] = 0u;
        }
        if (k < end) {
          T* y = head_at<T, I>(a.side[0].y, a.side[1].y, here, hq, k);
          if (a.pass)
            me.template store<true>(y, now[i]);
          else
            me.store(y, now[i]);
        }
      }
    }
  }
}

// The gradient.  A lane sums dgamma of its columns, for either side, in granules of
// its own in shared memory (in registers, with a change of sides at every token,
// fp32 4096x32+8x128 47.5 -> 52.3 us); a CTA's sums become its partial row.  The
// next heads of a group are in flight, over the ends of tokens, while one is at
// work.
template <typename D, int CA, bool PAIRS, int LANES>
struct HeadGradRing {
  using Lane = HeadLane<D, CA, PAIRS, 16 * LANES>;
  using T = typename D::T;
  static constexpr bool COPIES = sizeof(T) == 2 && CA >= 4;
  using Type = std::conditional_t<COPIES, CopyRing<Lane, T>, RegisterRing<Lane, T>>;
};
template <typename D, int CA, bool PAIRS, int LANES, typename I>
__global__ void __launch_bounds__(kHeadThreads, kHeadPerSm) head_rotary_grad_kernel(const HeadArgs a) {
  using Lane = HeadLane<D, CA, PAIRS, 16 * LANES>;
  using T = typename D::T;
  using Ring = typename HeadGradRing<D, CA, PAIRS, LANES>::Type;
  extern __shared__ __align__(16) float slots[];  // gamma of both sides, each warp's angles, sums and ring
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = LANES ? LANES : a.lanes;
  const int groups = 32 / lanes, group = lane / lanes, unit = lane & (lanes - 1);
  const Lane me(unit, a.D, a.R);
  const float inv_d = 1.f / (float)a.D;
  const int hq = a.side[0].heads, heads = hq + a.side[1].heads;
  const uint32_t gammas = smem_u32(slots + unit * kHeadSlot);
  float* angles = slots + (2 + warp) * lanes * kHeadSlot;
  const uint32_t angle = smem_u32(angles + unit * kHeadSlot);
  float4* sums = reinterpret_cast<float4*>(slots + (2 + kHeadWarps) * lanes * kHeadSlot);  // [warp][side][granule][lane]
  float4* mine = sums + warp * 256 + lane;
  Ring ring(reinterpret_cast<unsigned char*>(sums + kHeadWarps * 256) + warp * Ring::BYTES, lane, unit, lanes, a.D);
  pdl_launch_dependents();
  pdl_wait_primary();
  // the heads that are fetched, AHEAD units before those that are at work
  HeadShare share(a, blockIdx.x * kHeadWarps + warp), work = share;
  HeadToken token(a, share.first), ahead = token;
  const int tokens = share.left > 0 ? (int)((share.lo + share.left + a.its - 1) / a.its) : 0;
  HeadPlace<I> px(ahead, a.side[0].x, a.side[1].x, hq), py(ahead, a.side[0].dy, a.side[1].dy, hq);
  int fk = 0, fend = 0;  // the next head to fetch (of group 0), and the end of the token's
  bool first = true;
  auto fetch = [&] {
    if (fk >= fend) {
      int lo, hi;
      if (!share.take(a, lo, hi)) {
        ring.fetch(me, false, nullptr, nullptr);
        return;
      }
      if (!first) {
        ahead.step(a);
        px = HeadPlace<I>(ahead, a.side[0].x, a.side[1].x, hq);
        py = HeadPlace<I>(ahead, a.side[0].dy, a.side[1].dy, hq);
      }
      first = false;
      fk = lo * groups;
      fend = min(hi * groups, heads);
    }
    const int k = fk + group;
    ring.fetch(me, k < fend, head_at<T, I>(a.side[0].x, a.side[1].x, px, hq, k), head_at<T, I>(a.side[0].dy, a.side[1].dy, py, hq, k));
    fk += groups;
  };
#pragma unroll
  for (int i = 0; i < Ring::AHEAD; ++i) fetch();
  HeadAngles<D, LANES> way(a, angles, lane, token, tokens);
  for (int k = 0; k < 2; ++k)
    head_gamma<Lane, D>(slots + k * lanes * kHeadSlot, a, a.side[k].gamma, threadIdx.x, kHeadThreads);
#pragma unroll
  for (int j = 0; j < 8; ++j) mine[32 * j] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  int lo, hi;
  for (bool more = work.take(a, lo, hi); more; more = work.take(a, lo, hi)) {
    const HeadPlace<I> dst(token, a.side[0].y, a.side[1].y, hq);
    token.step(a);
    const int end = min(hi * groups, heads);
    const bool good = way.turn_over();
#pragma unroll 1
    for (int k = lo * groups + group; k - group < end; k += groups) {
      float2 p[4], q[4], u[4], v[4];
      {
        uint32_t wx[Lane::NW], wy[Lane::NW];
        ring.take(wx, wy);
        Lane::unpack(wx, p, q);
        Lane::unpack(wy, u, v);
      }
      fetch();
      const int which = k < hq ? 0 : 1;
      if (good) me.template turn<true>(u, v, angle);
      float2 sx = splat2(0.f), sw = splat2(0.f);
      const uint32_t gamma = gammas + which * lanes * kHeadSlot * 4;
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
      lanes_sum<2, LANES>(m, lanes);
      if (k >= end) continue;  // no lane exchanges anything below
      uint32_t o[Lane::NW];
      if (good) {
        const float r = rsqrtf(fmaf(m[0], inv_d, a.eps));
        // dx = rstd (w - x rstd^2 mean(w x)); w is formed again rather than kept
        const float2 r2 = splat2(r), k2 = splat2(-(m[1] * inv_d) * r * r);
        float4* at = mine + which * 128;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 x = at[32 * j], y = at[32 * (2 + j)];
          const float2 x0 = fma2(u[2 * j], mul2(p[2 * j], r2), make_float2(x.x, x.y));
          const float2 x1 = fma2(u[2 * j + 1], mul2(p[2 * j + 1], r2), make_float2(x.z, x.w));
          const float2 y0 = fma2(v[2 * j], mul2(q[2 * j], r2), make_float2(y.x, y.y));
          const float2 y1 = fma2(v[2 * j + 1], mul2(q[2 * j + 1], r2), make_float2(y.z, y.w));
          at[32 * j] = make_float4(x0.x, x0.y, x1.x, x1.y);
          at[32 * (2 + j)] = make_float4(y0.x, y0.y, y1.x, y1.y);
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
      me.store(head_at<T, I>(a.side[0].y, a.side[1].y, dst, hq, k), o);
    }
  }
  if (!a.want) return;
  __syncthreads();
  // column by column, over warps and groups in a fixed order
  for (int i = threadIdx.x; i < 2 * lanes * 16; i += kHeadThreads) {
    const int k = i / (lanes * 16), l = i / 16 % lanes, e = i % 16;
    float sum = 0.f;
    for (int w = 0; w < kHeadWarps; ++w)
      for (int g = 0; g < groups; ++g)
        sum += reinterpret_cast<const float*>(sums + (w * 2 + k) * 128 + e / 4 * 32 + g * lanes + l)[e % 4];
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

// Lanes a head takes: whole units of 16 columns, rounded to a power of two.
inline int head_lanes(const HeadArgs& a) {
  const int units = a.interleaved || a.R == 0 ? (a.D + 15) / 16 : (a.R / 2 + 7) / 8 + (a.D - a.R + 15) / 16;
  int lanes = 1;
  while (lanes < units) lanes <<= 1;
  return lanes;
}

// Columns an access: eight (16 bytes of half precision, 32 of fp32), four or one,
// whichever divides every column that an access starts at, and fits every tensor.
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
  return (bits & (8 * ES - 1)) == 0 ? 8 : (bits & (4 * ES - 1)) == 0 ? 4 : 1;
}

// The kernel on as many CTAs as are resident, or fewer.  Its units are shared out
// to the warps one by one: whole tokens would leave some warps with four and others
// with three of 8192 (56 us for 51.8).
template <typename K>
cudaError_t run_heads(K kern, HeadArgs& a, size_t smem, KernelMemo& memo, const DeviceInfo& dev, cudaStream_t s, int* ctas) {
  if (smem > 48 * 1024) {
    const cudaError_t e = memo.allow_smem(kern, dev.max_smem_optin - 1024, dev);
    if (e != cudaSuccess) return e;
  }
  const int resident = memo.resident(kHeadThreads, smem, dev, [&](int* n) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, kHeadThreads, smem);
    *n = std::min(*n, kHeadPerSm) * dev.sm_count;
    return e;
  });
  const int groups = 32 / a.lanes;
  a.its = (a.side[0].heads + a.side[1].heads + groups - 1) / groups;
  const int64_t units = a.N * a.its;
  *ctas = (int)std::min<int64_t>((units + kHeadWarps - 1) / kHeadWarps, resident);
  a.each = units / ((int64_t)*ctas * kHeadWarps);
  a.extra = units % ((int64_t)*ctas * kHeadWarps);
  FirstLaunch first(kHeadThreads, smem, s, 1);
  return first.launch((unsigned)*ctas, true, kern, a);
}

template <typename D, int CA, bool PAIRS, int LANES, typename I>
cudaError_t run_head_rotary(HeadArgs a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int U = sizeof(typename D::T) == 2 ? 2 : 1;  // 64 bytes of a lane
  // Heads that L2 will not hold until they are read again (a half of its 129 MB, the
  // inputs passing through the other) do not displace the inputs: bf16 32+8x128, 16384
  // tokens 59.8 -> 58.3 us, 16+16x64 25.3 -> 23.9.
  a.pass = a.N * (a.side[0].heads + a.side[1].heads) * a.D * (int64_t)sizeof(typename D::T) > 64000000;
  static KernelMemo memo;
  int ctas;
  return run_heads(head_rotary_kernel<D, CA, PAIRS, U, LANES, I>, a, sizeof(float) * (2 + kHeadWarps) * a.lanes * kHeadSlot, memo,
                   dev, s, &ctas);
}

template <typename D, int CA, bool PAIRS, int LANES, typename I>
cudaError_t run_head_rotary_grad(HeadArgs a, const DeviceInfo& dev, cudaStream_t s, int* ctas) {
  static KernelMemo memo;
  return run_heads(head_rotary_grad_kernel<D, CA, PAIRS, LANES, I>, a,
                   sizeof(float) * (2 + kHeadWarps) * a.lanes * kHeadSlot +
                       kHeadWarps * (4096 + HeadGradRing<D, CA, PAIRS, LANES>::Type::BYTES),
                   memo, dev, s, ctas);
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
cudaError_t head_variants(const HeadArgs& a, bool grad, F&& f) {
  const int access = head_access<D>(a, grad);
  auto with = [&](auto ca, auto l, auto off) {
    return a.interleaved && a.R ? f(ca, std::integral_constant<bool, true>{}, l, off)
                                : f(ca, std::integral_constant<bool, false>{}, l, off);
  };
  const std::integral_constant<int, 8> eight;
  const std::integral_constant<int, 4> four;
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 0> any;
  if (!head_offsets_fit(a, grad)) return access == 8 ? with(eight, any, int64_t{}) : with(one, any, int64_t{});
  if (access == 8 && a.R == a.D && a.D == 16 * a.lanes) {
    if (a.D == 64) return with(eight, std::integral_constant<int, 4>{}, uint32_t{});
    if (a.D == 128) return with(eight, std::integral_constant<int, 8>{}, uint32_t{});
    if (a.D == 256) return with(eight, std::integral_constant<int, 16>{}, uint32_t{});
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
