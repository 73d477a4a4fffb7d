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

constexpr int kLogprobThreads = 512;  // most of a CTA
constexpr int kLogprobMaxCluster = 8;
constexpr int kTopCandidates = 2048;
constexpr int kTopGroups = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;
// Differences this far down (in powers of two) are nothing beside 1; a product
// with one must stay finite.
constexpr float kFarDown = -1e4f;

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
  __device__ static __forceinline__ void fill(uint32_t (&w)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = kMasked;
  }
  // Columns [col, col + GE) of the row; -inf outside [0, V).
  __device__ static __forceinline__ void load(const T* row, int col, int V, uint32_t (&w)[8]) {
    if (col >= 0 && col + GE <= V) {
      ld_stream32(row + col, w);
      return;
    }
    fill(w);
#pragma unroll
    for (int e = 0; e < GE; ++e) {
      if (col + e >= 0 && col + e < V) {
        if constexpr (ES == 4) {
          w[e] = Chunk<D, ES, 4>::ldg32(row + col + e);
        } else {
          const uint32_t v = Chunk<D, ES, 4>::ldg16(row + col + e);
          w[e / 2] = e & 1 ? __byte_perm(w[e / 2], v, 0x5410) : __byte_perm(v, w[e / 2], 0x7610);
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

// Sort `n` keys in shared memory, largest first, with all threads of the CTA;
// those behind n up to the next power of two are overwritten.
__device__ __forceinline__ void sort_keys(unsigned long long* key, int n) {
  int size = 1;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += blockDim.x) key[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += blockDim.x) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const unsigned long long x = key[lo], y = key[hi];
        if ((x < y) == ((lo & k) == 0)) {
          key[lo] = y;
          key[hi] = x;
        }
      }
      __syncthreads();
    }
  }
}

__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v, int lanes) {
  for (int off = 1; off < lanes; off <<= 1) {
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

struct TopShared {
  unsigned long long key[kTopCandidates];
  unsigned long long group[kTopGroups];
  unsigned long long tau;
  int list[kLogprobThreads];
  int listed, found;
  unsigned long long best[kMaxTop];
};

// The first `top` keys of this CTA's chunks [first, last) into sh.best (0 where
// there are fewer).  Each thread comes with its largest logit and the chunk it
// met it in first.  A key at that chunk's last column is no larger than the key
// of the logit itself, so at least `top` logits reach tau, the top-th largest of
// those over groups of threads; all that do are in the chunks of threads whose
// own key does.  Only those chunks are read again (they are in L2): a 25th of the
// row for 20 of 512 threads.
template <typename D>
__device__ __forceinline__ void cta_top(TopShared& sh, const typename D::T* z, int a0, int V, int first, int last, int top,
                                        float mx, int mi) {
  using L = LogitChunk<D>;
  const int lane = threadIdx.x & 31;
  const float none = __int_as_float(0xff800000);
  const unsigned long long mine = mx > none ? top_key(mx, mi * L::GE - a0 + L::GE - 1) : 0ull;
  const int per = max(1, (int)blockDim.x / kTopGroups), groups = blockDim.x / per;
  if (threadIdx.x == 0) {
    sh.tau = 1ull;
    sh.listed = sh.found = 0;
  }
  const unsigned long long g = warp_max64(mine, per);
  if (lane % per == 0) sh.group[threadIdx.x / per] = g;
  __syncthreads();
  if (threadIdx.x < groups) {
    const unsigned long long k = sh.group[threadIdx.x];
    int rank = 0;
    for (int i = 0; i < groups; ++i) rank += sh.group[i] > k;
    if (k != 0 && rank == top - 1) sh.tau = k;
  }
  __syncthreads();
  const unsigned long long tau = sh.tau;
  if (mine >= tau) sh.list[atomicAdd(&sh.listed, 1)] = threadIdx.x;
  __syncthreads();
  const int each = (last - first + blockDim.x - 1) / blockDim.x;  // chunks a thread
  const int pairs = sh.listed * each;
  for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
    const int i = first + sh.list[p / each] + (p % each) * blockDim.x;
    if (i >= last) continue;
    uint32_t w[8];
    const int col = i * L::GE - a0;
    L::load(z, col, V, w);
#pragma unroll
    for (int e = 0; e < L::GE; ++e) {
      const float2 f = word_pair<D>(w, e / 2);
      const float v = e & 1 ? f.y : f.x;
      if (v > none) {
        const unsigned long long k = top_key(v, col + e);
        if (k >= tau) {
          const int at = atomicAdd(&sh.found, 1);
          if (at < kTopCandidates) sh.key[at] = k;
        }
      }
    }
  }
  __syncthreads();
  const int found = sh.found;
  if (found <= kTopCandidates) {
    sort_keys(sh.key, found);
    if (threadIdx.x < kMaxTop) sh.best[threadIdx.x] = threadIdx.x < min(found, top) ? sh.key[threadIdx.x] : 0ull;
    __syncthreads();
    return;
  }
  // More than fit (the largest logits crowd into few threads' chunks): one after
  // another, each the largest below the one before it.
  unsigned long long before = ~0ull;
  for (int r = 0; r < top; ++r) {
    unsigned long long best = 0;
    for (int i = first + threadIdx.x; i < last; i += blockDim.x) {
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
    best = warp_max64(best, 32);
    if (lane == 0) sh.group[threadIdx.x >> 5] = best;
    __syncthreads();
    for (int i = 0; i < (int)blockDim.x / 32; ++i) best = sh.group[i] > best ? sh.group[i] : best;
    if (threadIdx.x == 0) sh.best[r] = best;
    before = best;
    __syncthreads();
  }
}

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

// The whole row's sums in thread 0 (and its maximum in every thread).
__device__ __forceinline__ void cta_sums(RowSums& r, float c2, float (*red)[kLogprobThreads / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float m = r.mx;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (warps > 1) {
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
    m = lane < warps ? red[0][lane] : r.mx;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  }
  r.mx = m;
  r.move(fmaxf(m, kLowest), c2);
  float v[2] = {r.s, r.u};
  warp_sum<2>(v);
  if (warps > 1) {
    if (lane == 0) {
      red[1][warp] = v[0];
      red[2][warp] = v[1];
    }
    __syncthreads();
    v[0] = lane < warps ? red[1][lane] : 0.f;
    v[1] = lane < warps ? red[2][lane] : 0.f;
    warp_sum<2>(v);
  }
  r.s = v[0];
  r.u = v[1];
}

// One row a CTA, or a row a cluster of `cl`, whose CTAs take consecutive parts
// of its chunks.  U chunks of a thread are in flight at a time.
template <typename D, bool ENT, bool TOP>
__global__ void __launch_bounds__(kLogprobThreads, 2) logprob_kernel(const LogprobArgs a) {
  using L = LogitChunk<D>;
  using T = typename D::T;
  constexpr int U = 4;
  __shared__ float red[3][kLogprobThreads / 32];
  __shared__ float part_sums[3];
  __shared__ __align__(16) unsigned char top_raw[TOP ? sizeof(TopShared) : 16];
  TopShared& ts = *reinterpret_cast<TopShared*>(top_raw);
  pdl_launch_dependents();
  pdl_wait_primary();
  const int crank = a.cl > 1 ? (int)cluster_ctarank() : 0;
  const int64_t row = blockIdx.x / a.cl;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  const int a0 = L::lead(z);
  const int chunks = (a.V + a0 + L::GE - 1) / L::GE, part = (chunks + a.cl - 1) / a.cl;
  const int first = min(crank * part, chunks), last = min(first + part, chunks);
  const float c2 = a.scale * kLog2e;

  // the row's token, and its logit, for the end
  float zt = 0.f;
  int has = 0;
  if (crank == 0 && threadIdx.x == 0 && a.tokens) {
    const int64_t tok = a.tok64 ? reinterpret_cast<const long long*>(a.tokens)[row]
                                : (int64_t) reinterpret_cast<const int*>(a.tokens)[row];
    if (tok != a.ignore) {
      if (tok >= 0 && tok < a.V) {
        has = 1;
        zt = load_elem<D>(z, tok);
      } else {
        atomicOr(a.err, kErrBadToken);
      }
    }
  }

  const float none = __int_as_float(0xff800000);
  RowSums r{none, kLowest, 0.f, 0.f};
  float2 s2 = splat2(0.f), u2 = splat2(0.f);
  int mi = 0;
  for (int base = first + threadIdx.x; base < last; base += U * blockDim.x) {
    uint32_t w[U][8];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = base + k * blockDim.x;
      if (i < last) L::load(z, i * L::GE - a0, a.V, w[k]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (base + k * (int)blockDim.x >= last) break;
      const float cm = L::max(w[k]);
      if (TOP && cm > r.mx) mi = base + k * blockDim.x;
      r.mx = fmaxf(r.mx, cm);
      if ((cm - r.ref) * c2 > kSlack) {
        r.s = s2.x + s2.y;
        r.u = u2.x + u2.y;
        r.move(cm, c2);
        s2 = make_float2(r.s, 0.f);
        u2 = make_float2(r.u, 0.f);
      }
      const float2 ref2 = splat2(r.ref), cc = splat2(c2);
      float2 du = splat2(0.f);
#pragma unroll
      for (int j = 0; j < L::GE / 2; ++j) {
        const float2 x = mul2(sub2(word_pair<D>(w[k], j), ref2), cc);
        const float2 e = make_float2(ex2(x.x), ex2(x.y));
        s2 = add2(s2, e);
        if (ENT) du = fma2(e, x, du);
      }
      if (ENT) {
        if (isnan(du.x + du.y)) {  // a logit of -inf: 0 times its -inf counts as 0
          du = splat2(0.f);
#pragma unroll
          for (int j = 0; j < L::GE / 2; ++j) {
            const float2 x = mul2(sub2(word_pair<D>(w[k], j), ref2), cc);
            du = fma2(make_float2(ex2(x.x), ex2(x.y)), make_float2(fmaxf(x.x, kFarDown), fmaxf(x.y, kFarDown)), du);
          }
        }
        u2 = add2(u2, du);
      }
    }
  }
  r.s = s2.x + s2.y;
  r.u = u2.x + u2.y;
  const float my_max = r.mx;
  cta_sums(r, c2, red);
  if constexpr (TOP) cta_top<D>(ts, z, a0, a.V, first, last, a.top, my_max, mi);
  if (a.cl > 1) {
    if (threadIdx.x == 0) {
      part_sums[0] = r.mx;
      part_sums[1] = r.s;
      part_sums[2] = r.u;
    }
    cluster_sync_all();
    if (crank == 0) {
      if (threadIdx.x < 32) {
        const bool on = (int)threadIdx.x < a.cl;
        RowSums q{none, kLowest, 0.f, 0.f};
        if (on) {
          q.mx = cluster_ld_f32(&part_sums[0], threadIdx.x);
          q.s = cluster_ld_f32(&part_sums[1], threadIdx.x);
          q.u = cluster_ld_f32(&part_sums[2], threadIdx.x);
          q.ref = fmaxf(q.mx, kLowest);
        }
        float m = q.mx;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        q.move(fmaxf(m, kLowest), c2);
        float v[2] = {q.s, q.u};
        warp_sum<2>(v);
        r = RowSums{m, fmaxf(m, kLowest), v[0], v[1]};
      }
      if constexpr (TOP) {
        for (int i = threadIdx.x; i < a.cl * a.top; i += blockDim.x)
          ts.key[i] = cluster_ld_u64(&ts.best[i % a.top], (unsigned)(i / a.top));
      }
      __syncwarp();
    }
    cluster_sync_all();  // no CTA leaves, or writes its parts again, while they are read
    if (crank != 0) return;
    if constexpr (TOP) {
      __syncthreads();
      sort_keys(ts.key, a.cl * a.top);
      if (threadIdx.x < kMaxTop) ts.best[threadIdx.x] = threadIdx.x < a.top ? ts.key[threadIdx.x] : 0ull;
    }
  }
  const float log_sum = logf(r.s);  // 0 gives -inf
  if (threadIdx.x == 0) {
    if (a.stats) a.stats[row] = make_float2(r.mx, log_sum);
    if (a.lse) a.lse[row] = r.mx == none ? log_sum : fmaf(a.scale, r.mx, log_sum);
    // log 2 turns the sums of exponents of two into those of e
    if (ENT && a.entropy) a.entropy[row] = r.s == 0.f ? 0.f : log_sum - 0.6931471805599453f * (r.u / r.s);
    if (a.logprob) a.logprob[row] = !has ? 0.f : r.s == 0.f ? none : fmaf(a.scale, zt - r.mx, -log_sum);
  }
  if constexpr (TOP) {
    if (threadIdx.x == 0) {
      part_sums[0] = r.mx;
      part_sums[1] = log_sum;
    }
    __syncthreads();
    if ((int)threadIdx.x < a.top) {
      const unsigned long long k = ts.best[threadIdx.x];
      a.top_id[row * a.top + threadIdx.x] = k ? key_col(k) : -1;
      a.top_logprob[row * a.top + threadIdx.x] =
          k ? fmaf(a.scale, key_value(k) - part_sums[0], -part_sums[1]) : none;
    }
  }
}

// The gradient: tiles of U * tx chunks of one row, 256 / tx rows a CTA.  SAME:
// logits and gradient have the same lead, so that aligned chunks of the one are
// aligned in the other.
constexpr int kLogprobGradThreads = 256;
constexpr int kLogprobGradU = 2;
template <typename D, bool ENT, bool SAME>
__global__ void __launch_bounds__(kLogprobGradThreads, 4) logprob_grad_kernel(const LogprobGradArgs a) {
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
      if (tok != a.ignore) {
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
  // few rows: clusters share them, as long as a CTA keeps 256 chunks
  a.cl = 1;
  while (a.cl < kLogprobMaxCluster && a.N * a.cl * 2 <= 2 * (int64_t)dev.sm_count && chunks / (a.cl * 2) >= 256) a.cl *= 2;
  const int want = (chunks / a.cl + 3) / 4;
  int threads = 32;
  while (threads < kLogprobThreads && threads < want) threads *= 2;
  FirstLaunch first((unsigned)threads, 0, s, a.cl);
  return first.launch((unsigned)(a.N * a.cl), true, logprob_kernel<D, ENT, TOP>, a);
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
  const int chunks = (a.V + L::GE - 1) / L::GE + 1;  // of any lead
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
