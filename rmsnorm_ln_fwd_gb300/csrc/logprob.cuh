// Log probabilities of given tokens, with entropy and top alternatives, from
// rows of logits z, and the logits' gradient.  With a = scale, m = max z,
// x_j = a (z_j - m), l = log sum exp(x_j), p_j = exp(x_j - l):
//   logprob = x_t - l,  lse = a m + l,  entropy = l - sum p_j x_j,
//   dz_j = a (dlogprob (1[j = t] - p_j) + dlse p_j - dentropy p_j (log p_j + entropy)).
// Differences are formed before they are scaled, and m and l are kept apart: a
// row that is masked throughout with the type's lowest value is then uniform, as
// its formula says, where a m + l would lose l.
//
// An exponential and about five flops an element, so the traffic bounds both:
// the forward reads the logits once, the gradient reads and writes them once.
#pragma once

#include <algorithm>

#include "chunk.cuh"
#include "common.cuh"
#include "logprob.h"
#include "stream.h"

namespace normk {

// 256 threads a CTA (us, 4096x131072, 333x50001 and 16384x4096 bf16: 159, 13, 28;
// 128 threads 198, 14.7, 83).  The kernel comes in three shapes of chunks that a
// thread has in flight and CTAs an SM, by how many CTAs there are: 6 and 2 where two
// an SM hold them all, 4 and 3 (80 registers) where three take as many waves as four,
// else 3 and 4.  (us, as 3 and 4; 4 and 3; 6 and 2: 4096x131072 159; 169; 184,
// 640x131072 37.8; 34.2; 40, 333x50001 12.8; 11.1; 16.3, 150x50001 in clusters of two
// 9.2; 7.0; 6.4, 2000x4096 7.2; 6.2; 5.3.  Four chunks and four CTAs, 64 registers, 159,
// 13.5; two 167, 12.5.)
constexpr int kLogprobThreads = 256;  // of a CTA
constexpr int kLogprobPerSm = 4;      // CTAs
constexpr int kLogprobMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;
// Differences this far down (in powers of two) are nothing beside 1; a product
// with one must stay finite.
constexpr float kFarDown = -1e4f;

// Whether a row has no token.
__device__ __forceinline__ bool ignored(int64_t token, int64_t ignore) { return token == ignore && ignore != NORM_NO_IGNORE; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 bytes of a row: the columns of chunk i are [i*GE - a0, i*GE - a0 + GE), a0
// the elements between the row's first one and the 32-byte boundary before it,
// so that every chunk but the first and last of a row is one aligned access
// whatever the row's address.
template <typename D>
struct LogitChunk {
  using T = typename D::T;
  static constexpr int ES = (int)sizeof(T);
  static constexpr int GE = 32 / ES;
  static constexpr uint32_t kMasked = ES == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;

  __device__ static __forceinline__ int lead(const T* row) {
    return (int)((reinterpret_cast<uintptr_t>(row) & 31u) / ES);
  }
  // Columns [col, col + GE) of the row; -inf outside [0, V).  AGAIN: a chunk here and
  // there, which asks L2 for no more than itself.
  template <bool AGAIN = false>
  __device__ static __forceinline__ void load(const T* row, int col, int V, uint32_t (&w)[8]) {
    if (col >= 0 && col + GE <= V) {
      if constexpr (AGAIN)
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(row + col));
      else
        ld_stream32(row + col, w);
      return;
    }
    // A part of one: whole words (a chunk starts at 32 bytes) and a half at either end
    // (by elements, us: 16384x602 bf16 16.6 for 13.7).
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w[k] = kMasked;
      if constexpr (ES == 4) {
        if ((unsigned)(col + k) < (unsigned)V) w[k] = Chunk<D, ES, 4>::ldg32(row + col + k);
      } else {
        const int c = col + 2 * k;
        const bool lo = (unsigned)c < (unsigned)V, hi = (unsigned)(c + 1) < (unsigned)V;
        if (lo && hi) {
          w[k] = Chunk<D, ES, 4>::ldg32(row + c);
        } else if (lo || hi) {
          const uint32_t v = Chunk<D, ES, 4>::ldg16(row + c + (lo ? 0 : 1));
          w[k] = lo ? __byte_perm(v, kMasked, 0x5410) : __byte_perm(kMasked, v, 0x5410);
        }
      }
    }
  }
  // The largest of a chunk, NaN left out (unless there is nothing else).
  __device__ static __forceinline__ float max(const uint32_t (&w)[8]) {
    if constexpr (ES == 4) {
      float m = __uint_as_float(w[0]);
#pragma unroll
      for (int k = 1; k < 8; ++k) m = fmaxf(m, __uint_as_float(w[k]));
      return m;
    } else if constexpr (std::is_same<T, __half>::value) {
      __half2 m = *reinterpret_cast<const __half2*>(&w[0]);
#pragma unroll
      for (int k = 1; k < 8; ++k) m = __hmax2(m, *reinterpret_cast<const __half2*>(&w[k]));
      const float2 f = __half22float2(m);
      return fmaxf(f.x, f.y);
    } else {
      __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&w[0]);
#pragma unroll
      for (int k = 1; k < 8; ++k) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[k]));
      const float2 f = __bfloat1622float2(m);
      return fmaxf(f.x, f.y);
    }
  }
};

// Order of the alternatives: larger logits first, then lower columns.  Larger
// keys come first; no element has key 0.  (-0 and +0 are equal.)
__device__ __forceinline__ unsigned long long top_key(float v, int col) {
  const uint32_t b = __float_as_uint(v + 0.f);
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return ((unsigned long long)o << 32) | (0xffffffffu - (uint32_t)col);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int key_col(unsigned long long k) { return (int)(0xffffffffu - (uint32_t)k); }

// The threads of a row: `n` of them (whole warps, a power of two), thread `t`.
struct RowGroup {
  int n, t, bar;
  __device__ __forceinline__ void sync() const {
    if (n == 32)
      __syncwarp();
    else
      named_barrier(bar, n);
  }
};

// Sort `n` keys in shared memory, largest first; those behind n up to the next
// power of two are overwritten.
__device__ __forceinline__ void sort_keys(const RowGroup& g, unsigned long long* key, int n) {
  int size = 1;
  while (size < n) size <<= 1;
  for (int i = n + g.t; i < size; i += g.n) key[i] = 0;
  g.sync();
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = g.t; i < size / 2; i += g.n) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const unsigned long long x = key[lo], y = key[hi];
        if ((x < y) == ((lo & k) == 0)) {
          key[lo] = y;
          key[hi] = x;
        }
      }
      g.sync();
    }
  }
}

// Where a key goes among `n`: the number of larger ones.  Two keys a load and eight
// loads in flight; key is 16-byte aligned and holds zeros up to a multiple of 16.
__device__ __forceinline__ int key_rank(const unsigned long long* key, int n, unsigned long long k) {
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < n; i += 16) {
    ulonglong2 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = reinterpret_cast<const ulonglong2*>(key + i)[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) rank += (v[j].x > k) + (v[j].y > k);
  }
  return rank;
}

// The first `top` of `n` keys (different ones, or 0) into best, 0 where there are
// fewer; best is all zeros before.  Keys go to their ranks, which takes no barrier,
// as long as a thread has few of them (320 candidates of a row masked with one value,
// 256 threads: 13.0 us a call for 16.1 by sorting).
__device__ __forceinline__ void best_keys(const RowGroup& g, unsigned long long* key, int n, int top, unsigned long long* best) {
  if (n <= max(2 * g.n, 128)) {
    if (n + g.t < (n + 15) / 16 * 16) key[n + g.t] = 0ull;
    g.sync();
#pragma unroll 1
    for (int i = g.t; i < n; i += g.n) {
      const unsigned long long k = key[i];
      const int rank = key_rank(key, n, k);
      if (rank < top && k != 0) best[rank] = k;
    }
  } else {
    sort_keys(g, key, n);
    if (g.t < min(n, top)) best[g.t] = key[g.t];
  }
  g.sync();
}

__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, v, off);
    v = o > v ? o : v;
  }
  return v;
}

// What a thread knows of its columns: the largest, a reference no more than
// 2^kSlack under it, and relative to that the sums of the exponentials e and of
// e times their exponents (powers of two).
constexpr float kSlack = 8.f;
struct RowSums {
  float mx, ref, s, u;
  // Relative to another reference.
  __device__ __forceinline__ void move(float to, float c2) {
    const float d = fmaxf((ref - to) * c2, kFarDown);
    const float r = ex2(d);
    u = r * fmaf(d, s, u);
    s *= r;
    ref = to;
  }
};

// Shared memory of a row's alternatives.  512 candidates: a row that is constant,
// or masked with one value, has 16 columns of one thread for each alternative.
constexpr int kTopCandidates = 512;
constexpr int kTopOneGroup = 24;  // alternatives that one group of threads a lane does for
struct __align__(16) TopShared {
  unsigned long long key[kTopCandidates];
  unsigned long long best[kMaxTop];
  unsigned long long tau;
  int listed, found;
  unsigned char list[kLogprobThreads];
};
// Followed by each thread's largest key.
__host__ __device__ constexpr int top_bytes(int rows) { return rows * (int)sizeof(TopShared) + 8 * kLogprobThreads; }

// The first `top` keys of the chunks [first, last) into sh.best (0 where there
// are fewer).  Each thread comes with its largest logit and the chunk it met it
// in first.  A key at that chunk's last column is no larger than the key of the
// logit itself, so at least `top` logits reach tau, the top-th largest of those
// over 32 groups of threads (the same lane of each warp) or, of more than 24, over 64
// (the same lane of each other warp); all that do are in the chunks of threads whose
// own key does.  Only those chunks are read again: a 12th of the row for 20 of 256
// threads, most of them still in L2.  The first warp finds tau and lists the threads;
// what all warps do between a row's two reads costs the others their issue slots.
// (us, bf16: 1x131072 with 20 of them 7.6, without 3.5; 1024x131072 62; 45; with 32 of
// them 66, 93 by 32 groups; with 20 56 for 62 by 64, but 512x4096 6.5 for 6.0.  Every
// warp finding tau: 4096x32000 with one 69 for 66, 512x4096 6.2 for 5.3.)
template <typename D>
__device__ __forceinline__ void row_top(const RowGroup& g, TopShared& sh, unsigned long long* lanes, const typename D::T* z,
                                        int a0, int V, int first, int last, int top, float mx, int mi) {
  using L = LogitChunk<D>;
  const int lane = threadIdx.x & 31;
  const float none = __int_as_float(0xff800000);
  const unsigned long long mine = mx > none ? top_key(mx, mi * L::GE - a0 + L::GE - 1) : 0ull;
  if (g.t < kMaxTop) sh.best[g.t] = 0ull;
  if (g.t == 0) sh.found = 0;
  lanes[g.t] = mine;
  g.sync();
  if (g.t < 32) {
    constexpr int W = kLogprobThreads / 32;
    unsigned long long k[W], most[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < W; ++i) {
      k[i] = 32 * i < g.n ? lanes[32 * i + lane] : 0ull;
      most[i & 1] = k[i] > most[i & 1] ? k[i] : most[i & 1];
    }
    unsigned long long tau = 1ull;  // fewer groups than alternatives have a logit at all: any will do
    if (top <= kTopOneGroup || g.n == 32) {
      const unsigned long long v = most[0] > most[1] ? most[0] : most[1];
      int rank = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) rank += __shfl_sync(0xffffffffu, v, i) > v;
      const unsigned at = __ballot_sync(0xffffffffu, rank == top - 1 && v != 0);
      if (at) tau = __shfl_sync(0xffffffffu, v, __ffs(at) - 1);
    } else {
      int rank[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const unsigned long long x = __shfl_sync(0xffffffffu, most[0], i), y = __shfl_sync(0xffffffffu, most[1], i);
        rank[0] += (x > most[0]) + (y > most[0]);
        rank[1] += (x > most[1]) + (y > most[1]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned at = __ballot_sync(0xffffffffu, rank[j] == top - 1 && most[j] != 0);
        if (at) tau = __shfl_sync(0xffffffffu, most[j], __ffs(at) - 1);
      }
    }
    int n = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const unsigned in = __ballot_sync(0xffffffffu, k[i] >= tau);
      if (k[i] >= tau) sh.list[n + __popc(in & ((1u << lane) - 1u))] = (unsigned char)(32 * i + lane);
      n += __popc(in);
    }
    if (lane == 0) {
      sh.listed = n;
      sh.tau = tau;
    }
  }
  g.sync();
  const unsigned long long tau = sh.tau;
  const int each = (last - first + g.n - 1) / g.n;  // chunks a thread
  const int pairs = sh.listed * each;
  const float least = tau > 1ull ? key_value(tau) : none;
  for (int p = g.t; p < pairs; p += g.n) {
    const int i = first + sh.list[p / each] + (p % each) * g.n;
    if (i >= last) continue;
    uint32_t w[8];
    const int col = i * L::GE - a0;
    L::template load<true>(z, col, V, w);
    if (!(L::max(w) >= least)) continue;
#pragma unroll
    for (int e = 0; e < L::GE; ++e) {
      const float2 f = word_pair<D>(w, e / 2);
      const float v = e & 1 ? f.y : f.x;
      if (v >= least && v > none) {
        const unsigned long long k = top_key(v, col + e);
        if (k >= tau) {
          const int to = atomicAdd(&sh.found, 1);
          if (to < kTopCandidates) sh.key[to] = k;
        }
      }
    }
  }
  g.sync();
  if (sh.found <= kTopCandidates) {
    best_keys(g, sh.key, sh.found, top, sh.best);
    return;
  }
  // More than fit (the largest logits crowd into few threads' chunks): one after
  // another, each the largest below the one before it.
  unsigned long long before = ~0ull;
  for (int r = 0; r < top; ++r) {
    unsigned long long best = 0;
    for (int i = first + g.t; i < last; i += g.n) {
      uint32_t w[8];
      const int col = i * L::GE - a0;
      L::load(z, col, V, w);
#pragma unroll
      for (int e = 0; e < L::GE; ++e) {
        const float2 f = word_pair<D>(w, e / 2);
        const float v = e & 1 ? f.y : f.x;
        if (v > none) {
          const unsigned long long k = top_key(v, col + e);
          if (k < before && k > best) best = k;
        }
      }
    }
    best = warp_max64(best);
    if (lane == 0) lanes[g.t >> 5] = best;
    g.sync();
    for (int i = 0; i < g.n / 32; ++i) best = lanes[i] > best ? lanes[i] : best;
    if (g.t == 0) sh.best[r] = best;
    before = best;
    g.sync();
  }
}

// cluster_sync_all in its two halves.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ float cluster_ld_f32(const float* local, unsigned rank) {
  unsigned a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long cluster_ld_u64(const unsigned long long* local, unsigned rank) {
  unsigned a;
  unsigned long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// The sums over each eight lanes, in all of them.
__device__ __forceinline__ void eight_sums(RowSums& r, float c2) {
  r.ref = fmaxf(r.mx, kLowest);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) r.mx = fmaxf(r.mx, __shfl_xor_sync(0xffffffffu, r.mx, off));
  r.move(fmaxf(r.mx, kLowest), c2);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) {
    r.s += __shfl_xor_sync(0xffffffffu, r.s, off);
    r.u += __shfl_xor_sync(0xffffffffu, r.u, off);
  }
}

// The sums over a row's threads, in all of them.  red: 3 floats a warp.
__device__ __forceinline__ void row_sums(const RowGroup& g, RowSums& r, float c2, float* red) {
  const int lane = threadIdx.x & 31, warp = g.t >> 5, warps = g.n >> 5;
  float m = r.mx;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  r.mx = m;
  r.move(fmaxf(m, kLowest), c2);
  float v[2] = {r.s, r.u};
  warp_sum<2>(v);
  r.s = v[0];
  r.u = v[1];
  if (warps == 1) return;
  if (lane == 0) {
    red[3 * warp] = r.mx;
    red[3 * warp + 1] = r.s;
    red[3 * warp + 2] = r.u;
  }
  g.sync();
  // eight lanes take the warps' sums, and the others the same, so that all end
  // with the same bits
  const int from = lane & 7;
  const bool on = from < warps;
  r.mx = on ? red[3 * from] : __int_as_float(0xff800000);
  r.s = on ? red[3 * from + 1] : 0.f;
  r.u = on ? red[3 * from + 2] : 0.f;
  eight_sums(r, c2);
}

// A row for a.tpr threads, or for a cluster of a.cl CTAs, which take consecutive
// parts of its chunks.  U chunks of a thread are in flight at a time.
template <typename D, bool ENT, bool TOP, int U, int PER_SM>
__global__ void __launch_bounds__(kLogprobThreads, PER_SM) logprob_kernel(const LogprobArgs a) {
  using L = LogitChunk<D>;
  using T = typename D::T;
  static_assert(kLogprobThreads <= 256 && kLogprobMaxCluster <= 8, "eight sums");
  extern __shared__ __align__(16) unsigned char top_raw[];
  __shared__ float red[3 * kLogprobThreads / 32];
  __shared__ float part_sums[3];
  const int gid = threadIdx.x / a.tpr, rows = kLogprobThreads / a.tpr;
  const RowGroup g{a.tpr, (int)threadIdx.x - gid * a.tpr, 1 + gid};
  TopShared& ts = reinterpret_cast<TopShared*>(top_raw)[gid];
  unsigned long long* lanes = reinterpret_cast<unsigned long long*>(top_raw + rows * sizeof(TopShared)) + gid * a.tpr;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int crank = a.cl > 1 ? (int)cluster_ctarank() : 0;
  const int64_t row = a.cl > 1 ? blockIdx.x / a.cl : (int64_t)blockIdx.x * rows + gid;
  if (row >= a.N) return;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  const int a0 = L::lead(z);
  const int chunks = (a.V + a0 + L::GE - 1) / L::GE, part = (chunks + a.cl - 1) / a.cl;
  const int first = min(crank * part, chunks), last = min(first + part, chunks);
  const float c2 = a.scale * kLog2e;

  // the row's token, looked at when the row is through
  int64_t tok = a.ignore;
  if (g.t == 0 && a.tokens)
    tok = a.tok64 ? reinterpret_cast<const long long*>(a.tokens)[row] : (int64_t) reinterpret_cast<const int*>(a.tokens)[row];

  const float none = __int_as_float(0xff800000);
  RowSums r{none, kLowest, 0.f, 0.f};
  float2 s2 = splat2(0.f), u2 = splat2(0.f);
  int mi = 0;
  auto fetch = [&](uint32_t (&w)[U][8], int base) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = base + k * g.n;
      if (i < last) L::load(z, i * L::GE - a0, a.V, w[k]);
    }
  };
  auto take = [&](const uint32_t (&w)[U][8], int base) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (base + k * g.n >= last) break;
      const float cm = L::max(w[k]);
      if (TOP && cm > r.mx) mi = base + k * g.n;
      r.mx = fmaxf(r.mx, cm);
      if ((cm - r.ref) * c2 > kSlack) {
        r.s = s2.x + s2.y;
        r.u = u2.x + u2.y;
        r.move(cm, c2);
        s2 = make_float2(r.s, 0.f);
        u2 = make_float2(r.u, 0.f);
      }
      const float2 ref2 = splat2(r.ref), cc = splat2(c2);
#pragma unroll
      for (int j = 0; j < L::GE / 2; ++j) {
        const float2 x = mul2(sub2(word_pair<D>(w[k], j), ref2), cc);
        const float2 e = make_float2(ex2(x.x), ex2(x.y));
        s2 = add2(s2, e);
        // 0 times the -inf of a logit of -inf counts as 0
        if (ENT) u2 = fma2(e, make_float2(fmaxf(x.x, kFarDown), fmaxf(x.y, kFarDown)), u2);
      }
    }
  };
  for (int base = first + g.t; base < last; base += U * g.n) {
    uint32_t w[U][8];
    fetch(w, base);
    take(w, base);
  }
  r.s = s2.x + s2.y;
  r.u = u2.x + u2.y;
  const bool has = tok != a.ignore && tok >= 0 && tok < a.V;
  const float zt = has ? load_elem<D>(z, tok) : 0.f;  // comes in beside the sums
  if constexpr (TOP) row_top<D>(g, ts, lanes, z, a0, a.V, first, last, a.top, r.mx, mi);
  row_sums(g, r, c2, red + 3 * (gid * a.tpr / 32));
  if (a.cl > 1) {
    if (g.t == 0) {
      part_sums[0] = r.mx;
      part_sums[1] = r.s;
      part_sums[2] = r.u;
    }
    cluster_sync_all();
    if (crank == 0) {
      const int from = threadIdx.x & 7;
      const bool on = from < a.cl;
      r.mx = on ? cluster_ld_f32(&part_sums[0], from) : none;
      r.s = on ? cluster_ld_f32(&part_sums[1], from) : 0.f;
      r.u = on ? cluster_ld_f32(&part_sums[2], from) : 0.f;
      eight_sums(r, c2);
      if constexpr (TOP) {
        for (int i = g.t; i < a.cl * a.top; i += g.n) ts.key[i] = cluster_ld_u64(&ts.best[i % a.top], (unsigned)(i / a.top));
      }
      __syncwarp();
    }
    cluster_arrive();  // no CTA leaves while its part is read
    if (crank != 0) {
      cluster_wait();
      return;
    }
    if constexpr (TOP) {
      g.sync();
      if (g.t < kMaxTop) ts.best[g.t] = 0ull;
      best_keys(g, ts.key, a.cl * a.top, a.top, ts.best);
    }
  }
  const float log_sum = logf(r.s);  // 0 gives -inf
  if (g.t == 0) {
    if (a.stats) a.stats[row] = make_float2(r.mx, log_sum);
    if (a.lse) a.lse[row] = r.mx == none ? log_sum : fmaf(a.scale, r.mx, log_sum);
    // log 2 turns the sums of exponents of two into those of e
    if (ENT && a.entropy) a.entropy[row] = r.s == 0.f ? 0.f : log_sum - 0.6931471805599453f * (r.u / r.s);
    if (a.logprob && !has && !ignored(tok, a.ignore)) atomicOr(a.err, kErrBadToken);
    if (a.logprob) a.logprob[row] = !has ? 0.f : r.s == 0.f ? none : fmaf(a.scale, zt - r.mx, -log_sum);
  }
  if constexpr (TOP) {
    if (g.t < a.top) {
      const unsigned long long k = ts.best[g.t];
      a.top_id[row * a.top + g.t] = k ? key_col(k) : -1;
      a.top_logprob[row * a.top + g.t] = k ? fmaf(a.scale, key_value(k) - r.mx, -log_sum) : none;
    }
  }
  if (a.cl > 1) {
    __syncwarp();
    cluster_wait();
  }
}

// The gradient: tiles of U * tx chunks of one row, 128 / tx rows a CTA.  SAME:
// logits and gradient have the same lead, so that aligned chunks of the one are
// aligned in the other; else the gradient is stored by elements (4096x50257 bf16 of row
// stride 50304 into contiguous rows 1026 us, into rows of that stride 120).  (us,
// 4096x131072 bf16, 333x50001 bf16: 128 threads and three chunks 309, 12.2; two 333,
// 12.9; four 315, 12.1; 256 and three 313, 12.5; two 342, 13.6; one 382, 14.5; 512 and
// two 349, 15.4.)
constexpr int kLogprobGradThreads = 128;
constexpr int kLogprobGradU = 3;
template <typename D, bool ENT, bool SAME>
__global__ void __launch_bounds__(kLogprobGradThreads, 8) logprob_grad_kernel(const LogprobGradArgs a) {
  using L = LogitChunk<D>;
  using T = typename D::T;
  constexpr int U = kLogprobGradU;
  const int tx = a.tx, rows = kLogprobGradThreads / tx;
  const int x = threadIdx.x % tx, y = threadIdx.x / tx;
  const int64_t groups = (a.N + rows - 1) / rows;
  const float c2 = a.scale * kLog2e;
  pdl_launch_dependents();
  pdl_wait_primary();
  for (int64_t item = blockIdx.x; item < groups * a.tiles; item += gridDim.x) {
    const int64_t row = (item / a.tiles) * rows + y;
    const int tile = (int)(item % a.tiles);
    if (row >= a.N) continue;
    const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
    T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
    const int a0 = L::lead(z);
    const int chunks = (a.V + a0 + L::GE - 1) / L::GE;
    const int base = tile * U * tx + x;
    if (base >= chunks) continue;
    uint32_t w[U][8];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (base + k * tx < chunks) L::load(z, (base + k * tx) * L::GE - a0, a.V, w[k]);
    const float2 st = a.stats[row];
    const bool empty = st.y == __int_as_float(0xff800000);
    float dlp = 0.f;
    int token = -1;
    if (a.dlogprob) {
      const int64_t tok = a.tok64 ? reinterpret_cast<const long long*>(a.tokens)[row]
                                  : (int64_t) reinterpret_cast<const int*>(a.tokens)[row];
      if (!ignored(tok, a.ignore)) {
        if (tok >= 0 && tok < a.V) {
          token = (int)tok;
          dlp = a.dlogprob[row];
        } else if (x == 0 && tile == 0) {
          atomicOr(a.err, kErrBadToken);
        }
      }
    }
    const float dl = a.dlse ? a.dlse[row] : 0.f;
    const float de = ENT ? a.dentropy[row] : 0.f;
    // dz = p (k0 + k1 log2 p) + the token's
    const float k0 = a.scale * (dl - dlp - (ENT ? de * a.entropy[row] : 0.f));
    const float k1 = ENT ? -a.scale * de * 0.6931471805599453f : 0.f;
    const float2 m2 = splat2(st.x), cc = splat2(c2), l2 = splat2(-st.y * kLog2e), k02 = splat2(k0), k12 = splat2(k1);
    auto grad = [&](float2 v) {
      const float2 lp = fma2(sub2(v, m2), cc, l2);
      const float2 p = make_float2(ex2(lp.x), ex2(lp.y));
      // p = 0 has no gradient, though its log is -inf
      return mul2(p, ENT ? fma2(make_float2(fmaxf(lp.x, kFarDown), fmaxf(lp.y, kFarDown)), k12, k02) : k02);
    };
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = base + k * tx;
      if (i >= chunks) break;
      const int col = i * L::GE - a0;
      // (the first chunk of a row may begin before it: col < 0, which no token is)
      const bool here = token >= 0 && token >= col && token < col + L::GE;
      const float zt = here ? load_elem<D>(z, token) : 0.f;
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < L::GE / 2; ++j) {
        float2 g = grad(word_pair<D>(w[k], j));
        if (empty) g = splat2(0.f);
        pair_word<D>(o, j, g);
      }
      if (SAME && col >= 0 && col + L::GE <= a.V) {
        st_vec32(dz + col, o);
      } else {
#pragma unroll
        for (int e = 0; e < L::GE; ++e) {
          if (col + e >= 0 && col + e < a.V) {
            if constexpr (L::ES == 4)
              reinterpret_cast<uint32_t*>(dz)[col + e] = o[e];
            else
              reinterpret_cast<uint16_t*>(dz)[col + e] = (uint16_t)(o[e / 2] >> (16 * (e & 1)));
          }
        }
      }
      // the token's own logit, over what the chunk's store left there
      if (here)
        store_elem<D>(dz, token, empty ? 0.f : fmaf(a.scale, dlp, grad(splat2(zt)).x));
    }
  }
}

template <typename D, bool ENT, bool TOP>
cudaError_t run_logprob(LogprobArgs a, const DeviceInfo& dev, cudaStream_t s) {
  constexpr int GE = LogitChunk<D>::GE;
  const int chunks = a.V / GE + 1;
  // Few rows: clusters share them, the largest of which all fit at once on the GPU
  // (which the runtime knows: three clusters of eight an SM leave SMs unused), two CTAs
  // an SM before three and four.  Those of two, four and eight have at least half a
  // chunk a thread, one and two; the larger ones at more than two CTAs an SM, and any
  // with alternatives, which its CTAs have to merge, four.  Those of eight that merge
  // leave a quarter of the places free: as long as an earlier call's merge, they find
  // none (32x131072 with 20 alternatives, call after call, 13.4 us for 10.6 in clusters
  // of four).  (us, bf16, in order of the list below, then without a cluster; * does not
  // fit: 24x131072 5.2, 5.6, 6.0, 6.3, 6.6, 7.6, 8.4, 9.4, 11.4; with 20 alternatives 9.7,
  // 10.7, 10.1, 10.5, 10.6, 12.1, 13.1, 14.1, 16.3; 57x131072 9.7*, 10.0*, 7.5, 7.9,
  // 9.1, 9.2, 8.7, 10.9, 12.2; 112x131072 17.2*, 14.9*, 13.5*, 12.5*, 10.3, 10.7, 11.5,
  // 14.3, 14.5; 128x32000 13.2*, 10.5*, 7.7*, 7.8*, 5.9, 5.3, 6.1, 7.0, 7.5; 32x32000
  // with 20 alternatives 11.8*, 9.1, 7.4, 7.7, 7.6, 7.2, 7.1, 7.3, 6.9.)
  struct Plan {
    int cl, per_sm;
  };
  constexpr Plan plans[] = {{8, 2}, {8, 3}, {4, 2}, {4, 3}, {4, 4}, {2, 2}, {2, 3}, {2, 4}};
  constexpr int count = sizeof(plans) / sizeof(plans[0]);
  static KernelMemo memo[count];
  auto with_kernel = [&](int per_sm, auto&& f) {
    return per_sm == 2 ? f(logprob_kernel<D, ENT, TOP, 6, 2>)
                       : per_sm == 3 ? f(logprob_kernel<D, ENT, TOP, 4, 3>) : f(logprob_kernel<D, ENT, TOP, 3, kLogprobPerSm>);
  };
  a.cl = 1;
  int per_sm = 0;
  for (int i = 0; i < count && a.cl == 1; ++i) {
    const int cl = plans[i].cl, per = plans[i].per_sm;
    if (a.N * cl > per * (int64_t)dev.sm_count || (TOP && cl == 8 && per > 2)) continue;
    if (chunks / cl < (TOP || (cl > 2 && per > 2) ? 4 * kLogprobThreads : cl * kLogprobThreads / 4)) continue;
    FirstLaunch shape(kLogprobThreads, TOP ? top_bytes(1) : 0, s, cl);
    shape.cfg.gridDim.x = (unsigned)cl;
    const int fit = memo[i].resident(kLogprobThreads, shape.cfg.dynamicSmemBytes, dev, [&](int* n) {
      return with_kernel(per, [&](auto kern) { return cudaOccupancyMaxActiveClusters(n, kern, &shape.cfg); });
    });
    if (a.N > (TOP && cl == 8 ? fit * 3 / 4 : fit)) continue;
    a.cl = cl;
    per_sm = per;
  }
  // Otherwise as many threads as leave each three chunks, or, where one wave of CTAs
  // does not hold that many, fewer, with up to 16: what a row costs besides its logits
  // is the same for each warp.  (us, bf16, three and 16 chunks a thread: 320x4096 2.9,
  // 3.8; 640x8192 4.65, 5.4; 16384x4096 with 16, 8, 4 27.6, 33, 51.  With 20
  // alternatives, as this has it, and two chunks: 4096x4096 20.3, 39; 2048x8192 16.9,
  // 24; 512x4096 6.0, 6.4.)  More than 24 alternatives take two warps, which have a
  // thread for each (8192x1000 with 32 31.9 for 66, with 20 25.8 for 21.1).
  a.tpr = a.cl > 1 ? kLogprobThreads : 32;
  const int least = TOP && a.top > kTopOneGroup && chunks > 32 ? 64 : 32;
  while (a.tpr < kLogprobThreads && (a.tpr < least || a.tpr * 3 < chunks)) a.tpr *= 2;
  while (a.cl == 1 && a.tpr > least && chunks <= 16 * (a.tpr / 2) &&
         a.N * a.tpr > (int64_t)kLogprobPerSm * dev.sm_count * kLogprobThreads)
    a.tpr /= 2;
  const int rows = kLogprobThreads / a.tpr;
  FirstLaunch first(kLogprobThreads, TOP ? top_bytes(rows) : 0, s, a.cl);
  const int64_t ctas = a.cl > 1 ? a.N * a.cl : (a.N + rows - 1) / rows;
  if (per_sm == 0) {
    // the fewest waves, in the fewest CTAs an SM
    auto waves = [&](int per) { return (ctas + per * (int64_t)dev.sm_count - 1) / (per * (int64_t)dev.sm_count); };
    per_sm = waves(2) == 1 ? 2 : waves(3) == waves(kLogprobPerSm) ? 3 : kLogprobPerSm;
  }
  return with_kernel(per_sm, [&](auto kern) { return first.launch((unsigned)ctas, true, kern, a); });
}

template <typename D>
cudaError_t launch_logprob(LogprobArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  a.err = dev.err;
  if (a.top) return a.entropy ? run_logprob<D, true, true>(a, dev, s) : run_logprob<D, false, true>(a, dev, s);
  return a.entropy ? run_logprob<D, true, false>(a, dev, s) : run_logprob<D, false, false>(a, dev, s);
}

template <typename D>
cudaError_t launch_logprob_grad(LogprobGradArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();
  using L = LogitChunk<D>;
  a.err = dev.err;
  // a row's chunks: one more where rows do not begin at 32 bytes
  const bool leads = ((reinterpret_cast<uintptr_t>(a.z) | (a.N > 1 ? (uintptr_t)(a.ldz * (int64_t)sizeof(typename D::T)) : 0u)) & 31u) != 0;
  const int chunks = (a.V + L::GE - 1) / L::GE + leads;
  a.tx = 32;
  while (a.tx < kLogprobGradThreads && a.tx * kLogprobGradU < chunks) a.tx *= 2;
  a.tiles = (chunks + a.tx * kLogprobGradU - 1) / (a.tx * kLogprobGradU);
  const int rows = kLogprobGradThreads / a.tx;
  const int64_t items = (a.N + rows - 1) / rows * a.tiles;
  const bool same = ((reinterpret_cast<uintptr_t>(a.z) ^ reinterpret_cast<uintptr_t>(a.dz)) & 31u) == 0 &&
                    (a.N == 1 || (((a.ldz - a.lddz) * (int64_t)sizeof(typename D::T)) & 31) == 0);
  FirstLaunch first(kLogprobGradThreads, 0, s, 1);
  const unsigned grid = (unsigned)std::min<int64_t>(items, 1 << 30);
  if (a.dentropy)
    return same ? first.launch(grid, true, logprob_grad_kernel<D, true, true>, a)
                : first.launch(grid, true, logprob_grad_kernel<D, true, false>, a);
  return same ? first.launch(grid, true, logprob_grad_kernel<D, false, true>, a)
              : first.launch(grid, true, logprob_grad_kernel<D, false, false>, a);
}

}  // namespace normk
