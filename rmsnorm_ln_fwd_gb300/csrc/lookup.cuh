// Token lookup: rows of a table times a scale, with or without the first
// RMSNorm of the residual stream they start, and the table's gradient.
//
//   h_i = scale * table[token_i]               stored, rounded to the row dtype
//   y_i = h_i * rstd_i * gamma,  rstd_i = 1/sqrt(mean(h_i^2) + eps), from the fp32 h
//   dtable[v] = scale * sum over i with token_i = v of dh_i
//
// A token outside the table gives a row of zeros, takes no part in the
// gradient, and sets a bit of the device error word.

#pragma once

#include <algorithm>

#include "chunk.cuh"
#include "common.cuh"
#include "stream.h"

namespace normk {

constexpr int kLookupLoopThreads = 256;

// The token at position i, or -1 if it is not a row of the table.
__device__ __forceinline__ int64_t load_token(const void* tokens, int tok64, int64_t i, int64_t V, unsigned* err) {
  const int64_t t = tok64 ? reinterpret_cast<const int64_t*>(tokens)[i]
                          : (int64_t)reinterpret_cast<const int32_t*>(tokens)[i];
  if (t < 0 || t >= V) {
    if (err) atomicOr(err, kErrBadToken);
    return -1;
  }
  return t;
}

// Any width, stride and alignment: one CTA a row at a time.
template <typename D>
__global__ void __launch_bounds__(kLookupLoopThreads) lookup_loop_kernel(const LookupArgs a) {
  using T = typename D::T;
  constexpr int NW = kLookupLoopThreads / 32;
  __shared__ float sh[2 * NW];
  const int lane = threadIdx.x & 31, wig = threadIdx.x >> 5;
  const bool w_f32 = a.w_f32 != 0;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const int64_t tok = load_token(a.tokens, a.tok64, row, a.V, threadIdx.x == 0 ? a.err : nullptr);
    const T* src = reinterpret_cast<const T*>(a.table) + (tok < 0 ? 0 : tok) * a.ldt;
    T* h = reinterpret_cast<T*>(a.h) + row * a.ldh;
    float s[1] = {0.f};
    for (int j = threadIdx.x; j < a.H; j += kLookupLoopThreads) {
      const float v = tok < 0 ? 0.f : a.scale * load_elem<D>(src, j);
      store_elem<D>(h, j, v);
      s[0] = fmaf(v, v, s[0]);
    }
    if (a.y == nullptr) continue;
    group_sum<1>(s, sh, NW, wig, lane, 1, parity);
    parity ^= 1;
    const float rstd = rsqrtf(s[0] * (1.f / (float)a.H) + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    T* y = reinterpret_cast<T*>(a.y) + row * a.ldy;
    for (int j = threadIdx.x; j < a.H; j += kLookupLoopThreads) {
      const float v = tok < 0 ? 0.f : a.scale * load_elem<D>(src, j);
      store_elem<D>(y, j, v * rstd * (a.gamma ? load_param<D>(a.gamma, j, w_f32) : 1.f));
    }
  }
}

// Floats of the row sums' scratch in front of the parameter slots, which need
// 16-byte alignment.
__host__ __device__ inline int lookup_red_floats(int rpc, int tpr) { return (rpc * 2 * (tpr / 32) + 3) & ~3; }

// Register rows.  A row group of tpr threads, E columns a thread (chunk.cuh),
// walks rows row, row + stride, ...: the next row's columns are in flight while
// this one is scaled, reduced and written, and the token of the row after that,
// whose address they would otherwise wait for.
template <typename D, int GB, int E_, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) lookup_rows_kernel(const LookupArgs a, const int tpr) {
  using C = Chunk<D, GB, E_>;
  using T = typename D::T;
  constexpr int E = C::E, NP = C::NP, NW = C::NW;
  constexpr int SLOT = param_slot<E, 1>();
  extern __shared__ __align__(16) float sh_look[];
  const int rpc = blockDim.x / tpr;
  const int group = threadIdx.x / tpr;
  const int t = threadIdx.x - group * tpr;
  const int nw = tpr >> 5, wig = t >> 5, lane = threadIdx.x & 31;
  const int b = C::base(t), lim = a.H - b;
  const bool norm = a.y != nullptr;
  float* sh = sh_look + group * (2 * nw);
  float* slot = sh_look + lookup_red_floats(rpc, tpr) + t * SLOT;  // gamma, shared by the groups
  const uint32_t slot32 = smem_u32(slot);
  const int64_t step = (int64_t)gridDim.x * rpc;
  int64_t row = (int64_t)blockIdx.x * rpc + group;
  unsigned* err = t == 0 ? a.err : nullptr;
  auto token = [&](int64_t r) { return load_token(a.tokens, a.tok64, r, a.V, err); };
  uint32_t nx[NW];
  auto fetch = [&](int64_t tok) {
    C::load(reinterpret_cast<const T*>(a.table) + (tok < 0 ? 0 : tok) * a.ldt + b, tok < 0 ? 0 : lim, nx);
  };
  pdl_launch_dependents();
  pdl_wait_primary();
  int64_t tok2 = -1;  // the next row's
  if (row < a.N) {
    fetch(token(row));
    if (row + step < a.N) tok2 = token(row + step);
  }
  if (norm && group == 0) {
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = 1.f;
    C::scale_by_param(a.gamma, a.w_f32 != 0, b, lim, f);
    put_params<E>(slot, f);
  }
  __syncthreads();
  T* hp = reinterpret_cast<T*>(a.h) + row * a.ldh + b;
  T* yp = norm ? reinterpret_cast<T*>(a.y) + row * a.ldy + b : nullptr;
  const int64_t hstep = step * a.ldh, ystep = step * a.ldy;
  const float2 scale2 = splat2(a.scale);
  const float inv_h = 1.f / (float)a.H;
  int parity = 0;
  for (; row < a.N; row += step, hp += hstep) {
    float2 f[NP], s2 = splat2(0.f);
    uint32_t out[NW];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      f[p] = mul2(word_pair<D>(nx, p), scale2);
      s2 = fma2(f[p], f[p], s2);
      pair_word<D>(out, p, f[p]);
    }
    if (row + step < a.N) {
      fetch(tok2);
      if (row + 2 * step < a.N) tok2 = token(row + 2 * step);
    }
    C::store(hp, lim, out);
    if (!norm) continue;
    float s[1] = {s2.x + s2.y};
    group_sum<1>(s, sh, nw, wig, lane, 1 + group, parity);
    parity ^= 1;
    const float rstd = rsqrtf(s[0] * inv_h + a.eps);
    if (t == 0 && a.rstd) a.rstd[row] = rstd;
    const float2 r2 = splat2(rstd);
#pragma unroll
    for (int q = 0; q < NP / 2; ++q) {
      float2 g[2];
      lds_pairs(slot32 + 16 * q, g);
#pragma unroll
      for (int i = 0; i < 2; ++i) pair_word<D>(out, 2 * q + i, mul2(mul2(f[2 * q + i], r2), g[i]));
    }
    C::store(yp, lim, out);
    yp += ystep;
  }
}

template <typename D, int GB, int E, int MAXT, int MINB>
static cudaError_t run_lookup_rows(const LookupArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  auto kern = lookup_rows_kernel<D, GB, E, MAXT, MINB>;
  const int tpr = chunk_threads(a.H, E);
  const int rpc = tpr <= 256 ? 256 / tpr : 1, threads = rpc * tpr;
  const size_t smem = sizeof(float) * ((size_t)lookup_red_floats(rpc, tpr) + (size_t)tpr * param_slot<E, 1>());
  static KernelMemo memo;
  if (smem > 48 * 1024) {
    cudaError_t e = memo.allow_smem(kern, dev.max_smem_optin - 1024, dev);
    if (e != cudaSuccess) return e;
  }
  const int per_sm = memo.resident(threads, smem, dev, [&](int* n) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, threads, smem);
  });
  const int64_t blocks = std::min<int64_t>((a.N + rpc - 1) / rpc, (int64_t)per_sm * dev.sm_count);
  FirstLaunch first((unsigned)threads, smem, s, 1);
  return first.launch((unsigned)blocks, true, kern, a, tpr);
}

// 32 bytes a thread up to 1024 threads, in fp32 64 bytes beyond.
template <typename D, int GB>
static cudaError_t run_lookup(const LookupArgs& a, const DeviceInfo& dev, cudaStream_t s, bool* done) {
  constexpr int E = 32 / (int)sizeof(typename D::T);
  *done = true;
  const int tpr = chunk_threads(a.H, E);
  // four CTAs an SM hold their registers to 64, which element by element spills
  // (16384x4096 bf16 with the norm 63.2 -> 58.9 us; 8192x2057 fp16 26.8 -> 41.5)
  if (tpr <= 256) return run_lookup_rows<D, GB, E, 256, (GB >= 16 ? 4 : 3)>(a, dev, s);
  if (tpr <= 1024) return run_lookup_rows<D, GB, E, 1024, 1>(a, dev, s);
  if constexpr (D::VEC == 4) {
    constexpr int GB2 = GB == 32 ? 16 : GB;
    if (chunk_threads(a.H, 16) <= 1024) return run_lookup_rows<D, GB2, 16, 1024, 1>(a, dev, s);
  }
  *done = false;
  return cudaSuccess;
}

template <typename D>
cudaError_t launch_lookup(LookupArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  using T = typename D::T;
  a.err = dev.err;
  if (dev.path != PATH_LOOP) {
    GranuleRule rule;
    rule.add(a.table, a.ldt, sizeof(T));
    rule.add(a.h, a.ldh, sizeof(T));
    if (a.y) rule.add(a.y, a.ldy, sizeof(T));
    const int gb = rule.bytes(a.H, sizeof(T));
    bool done = false;
    cudaError_t e = gb == 32   ? run_lookup<D, 32>(a, dev, s, &done)
                    : gb == 16 ? run_lookup<D, 16>(a, dev, s, &done)
                               : run_lookup<D, (int)sizeof(T)>(a, dev, s, &done);
    if (done) return e;
  }
  const int64_t blocks = std::min<int64_t>(a.N, (int64_t)dev.sm_count * 8);
  lookup_loop_kernel<D><<<(unsigned)blocks, kLookupLoopThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// The table's gradient.
//
// Kernel 1 sorts the tokens by id, stably, on one cluster of eight CTAs.  The
// rows that no token names are cleared (not when the gradient accumulates) by
// CTAs of kernel 3, which start beside the sort and go on beside the sums:
// clearing alone is all writes, which run at 0.86 of the copy rate (5.85 TB/s
// measured), and beside it the sums' reads come almost free.  For that they mark
// the ids of their range of rows from the tokens themselves; where that would
// cost more than it spares (short rows, or very many tokens) kernel 2, launched
// beside the sort, clears every row before kernel 3 begins, and ends after the
// sort, so that waiting for it is waiting for both.
// Kernel 3 takes the sorted tokens in tiles: a
// tile sums the gradient rows of each id in it, in position order, and stores
// the ids whose tokens all lie in the tile; the first and the last id of a tile
// may have tokens in its neighbours, and leave one partial row each.  Kernel 4
// sums the partial rows of those ids in tile order.  Every sum therefore has
// one order, whatever runs first: the gradient is the same bits at every call.
// ---------------------------------------------------------------------------

// Sort: a least-significant-digit radix sort of (id, position) pairs, ids
// 0..V with V for ignored tokens, `bits` a digit.  The cluster's 256 warps own
// equal contiguous parts of the input; a pass counts each warp's digits in
// shared memory, adds the counts up over warps and (through distributed shared
// memory) CTAs into each warp's first place for each digit, and moves the
// pairs in order, lanes of a digit ranked by a match across the warp, so equal
// ids keep their order (only the counting uses atomics, whose order is lost in
// the count).
constexpr int kSortCluster = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortMaxBits = 9;

struct SortPlan {
  int passes, bits;
};
inline SortPlan sort_plan(int64_t V) {
  int total = 1;
  while ((int64_t(1) << total) <= V) ++total;  // ids 0..V
  SortPlan p;
  p.passes = (total + kSortMaxBits - 1) / kSortMaxBits;
  p.bits = (total + p.passes - 1) / p.passes;
  return p;
}

__device__ __forceinline__ int ld_cluster_int(const int* local, unsigned rank) {
  unsigned addr;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// K > 0: a warp's part is at most 32*K items, which its lanes hold from the
// count to the move; K = 0: any length, read twice.
template <int K>
__device__ __forceinline__ void sort_tokens(const LookupGradArgs& a, SortPlan plan, int* smem) {
  constexpr int NWARP = kSortThreads / 32;
  const int bins = 1 << plan.bits;
  int* count = smem;                    // [warp][bin]
  int* total = count + NWARP * bins;    // [bin], this CTA's
  int* base = total + bins;             // [bin], first place of this CTA's digits
  int* wsum = base + bins;              // [warp]
  const unsigned rank = cluster_ctarank();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t part = ((a.N + kSortCluster * NWARP - 1) / (kSortCluster * NWARP) + 31) / 32 * 32;
  const int64_t lo = min(a.N, (int64_t)(rank * NWARP + w) * part), hi = min(a.N, lo + part);
  const unsigned below = (1u << lane) - 1u;
  int* mine = count + w * bins;
  uint2* src = nullptr;
  for (int pass = 0; pass < plan.passes; ++pass) {
    // the last pass ends in a.sorted
    uint2* dst = ((plan.passes - 1 - pass) & 1) ? a.other : a.sorted;
    const int shift = pass * plan.bits;
    auto fetch = [&](int64_t i) {
      if (pass > 0) return __ldcg(src + i);
      int64_t t = load_token(a.tokens, a.tok64, i, a.V, a.err);
      if (t < 0 || t == a.padding) t = a.V;
      return make_uint2((unsigned)t, (unsigned)i);
    };
    auto digit = [&](uint2 kv) { return (int)((kv.x >> shift) & (unsigned)(bins - 1)); };
    uint2 held[K > 0 ? K : 1];
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (lo + 32 * k + lane < hi) held[k] = fetch(lo + 32 * k + lane);
    }
    for (int b = lane; b < bins; b += 32) mine[b] = 0;
    __syncwarp();
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (lo + 32 * k + lane < hi) atomicAdd(&mine[digit(held[k])], 1);
    } else {
      for (int64_t i = lo + lane; i < hi; i += 32) atomicAdd(&mine[digit(fetch(i))], 1);
    }
    __syncthreads();
    // per bin: exclusive prefix over this CTA's warps, and its total
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
      int sum = 0;
#pragma unroll 8
      for (int k = 0; k < NWARP; ++k) {
        const int c = count[k * bins + b];
        count[k * bins + b] = sum;
        sum += c;
      }
      total[b] = sum;
    }
    cluster_sync_all();  // every CTA's totals are there
    int all = 0, before = 0;
    if (threadIdx.x < bins) {
#pragma unroll
      for (unsigned r = 0; r < kSortCluster; ++r) {
        const int c = ld_cluster_int(total + threadIdx.x, r);
        all += c;
        if (r < rank) before += c;
      }
    }
    // exclusive prefix of `all` over the bins (at most 512: threads of the first warps)
    int incl = all;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) wsum[w] = incl;
    __syncthreads();
    if (threadIdx.x < bins) {
      int first = incl - all + before;
      for (int k = 0; k < w; ++k) first += wsum[k];
      base[threadIdx.x] = first;
    }
    __syncthreads();
    auto move = [&](bool on, uint2 kv) {
      const unsigned act = __ballot_sync(0xffffffffu, on);
      int d = 0;
      unsigned same = 0u;
      if (on) {
        d = digit(kv);
        same = __match_any_sync(act, d);
        dst[base[d] + mine[d] + __popc(same & below)] = kv;
      }
      __syncwarp();  // every lane has read its counter
      if (on && (same & below) == 0) mine[d] += __popc(same);
      __syncwarp();
    };
    if constexpr (K > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (lo + 32 * k < hi) move(lo + 32 * k + lane < hi, held[k]);
    } else {
      for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const bool on = i0 + lane < hi;
        move(on, on ? fetch(i0 + lane) : make_uint2(0u, 0u));
      }
    }
    src = dst;
    cluster_sync_all();  // the pass's pairs are visible, its totals read
  }
}

// Kernel 1.  Launched without programmatic serialization: the clearing CTAs
// behind it write the table before they wait, so all that came before the call
// has to be through when this kernel starts.
static __global__ void __launch_bounds__(kSortThreads) lookup_grad_sort_kernel(const LookupGradArgs a, const SortPlan plan) {
  extern __shared__ __align__(16) int smem_sort[];
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.owners[0] = make_int2(0, 0);
  constexpr int64_t kWarps = kSortCluster * kSortThreads / 32;
  if (a.N <= kWarps * 32)
    sort_tokens<1>(a, plan, smem_sort);
  else if (a.N <= kWarps * 32 * 4)
    sort_tokens<4>(a, plan, smem_sort);
  else if (a.N <= kWarps * 32 * 8)
    sort_tokens<8>(a, plan, smem_sort);
  else
    sort_tokens<0>(a, plan, smem_sort);
}

constexpr int kClearThreads = 128;
constexpr int kClearMaxRange = 8192;  // rows a CTA marks at a time
// Clearing CTAs an SM (measured beside the sums, 16384 tokens into 131072x4096
// bf16, us: 1: 251, 2: 227, 3: 231, 4: 208, 6: 212, 8: 224, 12: 245).
constexpr int kClearPerSm = 4;
constexpr int kClearZeros = 8192;     // bytes of zeros in shared memory, the source of its copies

// Bulk copy from shared to global memory (both 16-byte aligned, bytes a
// multiple of 16), and the wait for this thread's copies to be written.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_s2g_drain() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

struct ClearSmem {
  unsigned marks[kClearMaxRange / 32];
  unsigned char zeros[kClearZeros];
};

// Clear part `part` of `parts` of the table's rows: those no token names
// (a.mark), or all.
template <typename O>
__device__ __forceinline__ void clear_rows(const LookupGradArgs& a, ClearSmem& sm, int part, int parts) {
  using T = typename O::T;
  const int nt = blockDim.x;
  for (int i = threadIdx.x; i < kClearZeros / 16; i += nt)
    reinterpret_cast<uint4*>(sm.zeros)[i] = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the __syncthreads below orders it for every thread)
  T* out = reinterpret_cast<T*>(a.dtable);
  const size_t row_bytes = (size_t)a.H * sizeof(T);
  const size_t bits = reinterpret_cast<uintptr_t>(out) | (size_t)a.lddt * sizeof(T) | row_bytes;
  int64_t lo, hi;
  cta_rows(a.V, part, parts, lo, hi);
  __syncthreads();
  if (!a.mark && (bits & 15u) == 0 && a.lddt == a.H) {  // one stretch of memory
    unsigned char* p = reinterpret_cast<unsigned char*>(out + lo * a.H);
    const int64_t bytes = (hi - lo) * (int64_t)row_bytes;
    for (int64_t i = (int64_t)threadIdx.x * kClearZeros; i < bytes; i += (int64_t)nt * kClearZeros)
      bulk_s2g(p + i, sm.zeros, (uint32_t)min(bytes - i, (int64_t)kClearZeros));
    lo = hi;
  }
  for (int64_t v0 = lo; v0 < hi; v0 += kClearMaxRange) {
    const int n = (int)min(hi - v0, (int64_t)kClearMaxRange);
    __syncthreads();
    for (int i = threadIdx.x; i < (n + 31) / 32; i += nt) sm.marks[i] = 0u;
    __syncthreads();
    if (a.mark) {
      auto mark = [&](int64_t t) {
        const int64_t at = t - v0;
        if (t >= 0 && t < a.V && t != a.padding && at >= 0 && at < n) atomicOr(&sm.marks[at >> 5], 1u << (at & 31));
      };
      // 16 bytes of tokens at a time where they are aligned, then the rest
      const int per = a.tok64 ? 2 : 4;
      const int64_t groups = (reinterpret_cast<uintptr_t>(a.tokens) & 15u) == 0 ? a.N / per : 0;
#pragma unroll 8
      for (int64_t i = threadIdx.x; i < groups; i += nt) {
        const uint4 u = ld_cached(reinterpret_cast<const uint4*>(a.tokens) + i);
        if (a.tok64) {
          mark((int64_t)(((unsigned long long)u.y << 32) | u.x));
          mark((int64_t)(((unsigned long long)u.w << 32) | u.z));
        } else {
          mark((int)u.x);
          mark((int)u.y);
          mark((int)u.z);
          mark((int)u.w);
        }
      }
      for (int64_t i = groups * per + threadIdx.x; i < a.N; i += nt)
        mark(load_token(a.tokens, a.tok64, i, a.V, nullptr));
      __syncthreads();
    }
    if ((bits & 15u) == 0) {
      // a thread a row, in bulk copies of the zeros
      for (int r = threadIdx.x; r < n; r += nt) {
        if ((sm.marks[r >> 5] >> (r & 31)) & 1u) continue;
        unsigned char* row = reinterpret_cast<unsigned char*>(out + (v0 + r) * a.lddt);
        for (size_t i = 0; i < row_bytes; i += kClearZeros)
          bulk_s2g(row + i, sm.zeros, (uint32_t)min(row_bytes - i, (size_t)kClearZeros));
      }
    } else {
      for (int r = threadIdx.x >> 5; r < n; r += nt / 32) {
        if ((sm.marks[r >> 5] >> (r & 31)) & 1u) continue;
        T* row = out + (v0 + r) * a.lddt;
        for (int j = threadIdx.x & 31; j < a.H; j += 32) row[j] = T(0.f);
      }
    }
  }
  bulk_s2g_drain();
}

// Kernel 2 (where rows are not marked).
template <typename O>
__global__ void __launch_bounds__(kClearThreads) lookup_grad_clear_kernel(const LookupGradArgs a) {
  __shared__ __align__(16) ClearSmem sm;
  pdl_launch_dependents();
  clear_rows<O>(a, sm, blockIdx.x, gridDim.x);
  pdl_wait_primary();  // the sort
}

// Store `v`, the sums of the thread's columns from column c of row `id`, times
// the scale, onto what the row holds when the gradient accumulates.  `vec`: the
// table allows 16-byte access.
template <typename O, typename C>
__device__ __forceinline__ void store_grad(const LookupGradArgs& a, int64_t id, int c, int lim, bool vec,
                                           const float (&v)[C::E]) {
  using T = typename O::T;
  T* row = reinterpret_cast<T*>(a.dtable) + id * a.lddt + c;
  constexpr int VEC = O::VEC;
  if constexpr (C::GE >= VEC) {
    if (vec) {
#pragma unroll
      for (int e = 0; e < C::E; e += VEC) {
        if (C::col(e) >= lim) continue;
        float f[VEC];
        if (a.accumulate) unpack<O>(ld_cached(row + C::col(e)), f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = fmaf(a.scale, v[e + i], a.accumulate ? f[i] : 0.f);
        st_vec(row + C::col(e), pack<O>(f));
      }
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < C::E; ++e) {
    if (C::col(e) >= lim) continue;
    store_elem<O>(row, C::col(e), fmaf(a.scale, v[e], a.accumulate ? load_elem<O>(row, C::col(e)) : 0.f));
  }
}

// Kernel 3: the first a.clearers CTAs clear rows; the others take tiles of
// sorted tokens by blocks of columns, 32 bytes a thread.  The rows' addresses
// come from the sorted pairs, so kTileBatch rows' loads are in flight at a time.
constexpr int kTileThreads = kClearThreads;
constexpr int kTileBatch = 8;

template <typename D, typename O, int GB>
__global__ void __launch_bounds__(kTileThreads) lookup_grad_tile_kernel(const LookupGradArgs a, int vec) {
  using C = Chunk<D, GB, 32 / (int)sizeof(typename D::T)>;
  using T = typename D::T;
  constexpr int E = C::E, NP = C::NP, NW = C::NW;
  const int nt = blockDim.x;
  __shared__ __align__(16) ClearSmem sm;
  __shared__ uint2 kv[kLookupMaxTile + 2];  // with the neighbours' nearest ids
  pdl_launch_dependents();
  if ((int)blockIdx.x < a.clearers) {
    clear_rows<O>(a, sm, blockIdx.x, a.clearers);
    pdl_wait_primary();
    return;
  }
  pdl_wait_primary();
  const unsigned tile = (blockIdx.x - a.clearers) / a.col_blocks, col_block = (blockIdx.x - a.clearers) % a.col_blocks;
  const int64_t first = (int64_t)tile * a.tile;
  const int n = (int)min((int64_t)a.tile, a.N - first);
  const unsigned none = 0xffffffffu;  // no id (ids are at most V < 2^31)
  for (int i = threadIdx.x; i < n + 2; i += nt) {
    const int64_t at = first + i - 1;
    kv[i] = at >= 0 && at < a.N ? __ldcg(a.sorted + at) : make_uint2(none, 0u);
  }
  __syncthreads();
  const unsigned ignored = (unsigned)a.V;
  const bool open_front = kv[0].x == kv[1].x;
  for (int c0 = col_block * (nt * E); c0 < a.H; c0 += a.col_blocks * (nt * E)) {
    const int c = c0 + C::base(threadIdx.x), lim = a.H - c;
    const T* src = reinterpret_cast<const T*>(a.dh) + c;
    float2 acc[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) acc[p] = splat2(0.f);
    uint32_t w[kTileBatch][NW];
    auto fetch = [&](int i, uint32_t (&into)[NW]) {
      const uint2 e = kv[min(i, n - 1) + 1];
      C::load(src + (int64_t)e.y * a.lddh, i < n && e.x != ignored ? lim : 0, into);
    };
#pragma unroll
    for (int k = 0; k < kTileBatch; ++k) fetch(k, w[k]);
    for (int i0 = 0; i0 < n; i0 += kTileBatch) {
#pragma unroll
      for (int k = 0; k < kTileBatch; ++k) {
        const int i = i0 + k;
        if (i >= n) break;
        const unsigned id = kv[i + 1].x;
        if (id == ignored) break;  // ignored tokens sort last
#pragma unroll
        for (int p = 0; p < NP; ++p) acc[p] = add2(acc[p], word_pair<D>(w[k], p));
        if (i + kTileBatch < n) fetch(i + kTileBatch, w[k]);
        if (i + 1 < n && kv[i + 2].x == id) continue;  // its last token in the tile
        float v[E];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          v[2 * p] = acc[p].x;
          v[2 * p + 1] = acc[p].y;
          acc[p] = splat2(0.f);
        }
        const bool front = open_front && id == kv[1].x, back = i + 1 == n && kv[n + 1].x == id;
        if (back && !front && c0 == 0 && threadIdx.x == 0) a.owners[atomicAdd(&a.owners[0].x, 1) + 1] = make_int2((int)tile, (int)id);
        if (front || back) {
          float* part = a.partial + ((size_t)2 * tile + (front ? 0 : 1)) * a.Hp + c;
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (C::col(e) < lim) part[C::col(e)] = v[e];
        } else {
          store_grad<O, C>(a, id, c, lim, vec != 0, v);
        }
      }
    }
  }
}

// Kernel 4: the ids whose tokens cross tiles.  Each is listed once, by the tile
// it begins in (in whatever order: they do not meet).  A CTA takes one after
// another and sums its partial rows over 256 columns (blockIdx.y): four row
// groups of 64 lanes, four columns a lane, each group every fourth row, eight
// loads in flight; then the groups in order.
constexpr int kJoinThreads = 256;
constexpr int kJoinLanes = 64;

template <typename O>
__global__ void __launch_bounds__(kJoinThreads) lookup_grad_join_kernel(const LookupGradArgs a) {
  constexpr int G = kJoinThreads / kJoinLanes, U = 8;
  pdl_wait_primary();
  __shared__ float4 sums[G - 1][kJoinLanes];
  const int64_t tile = a.tile, tiles = (a.N + tile - 1) / tile;
  const int g = threadIdx.x / kJoinLanes, lane = threadIdx.x % kJoinLanes;
  const int listed = __ldcg(&a.owners[0].x);
  for (int o = blockIdx.x; o < listed; o += gridDim.x) {
    const int2 owner = __ldcg(a.owners + 1 + o);
    const int64_t b = owner.x;
    const unsigned id = (unsigned)owner.y;
    // the id's tiles: b, and those after it that begin with it
    int64_t more = 0;
    for (int64_t t = b + 1;; t += kJoinThreads) {
      const int64_t at = t + threadIdx.x;
      const int c = __syncthreads_count(at < tiles && __ldcg(a.sorted + at * tile).x == id);
      more += c;
      if (c < kJoinThreads) break;
    }
    for (int c0 = blockIdx.y * (4 * kJoinLanes); c0 < a.Hp; c0 += gridDim.y * (4 * kJoinLanes)) {
      const int c = c0 + lane * 4;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < a.Hp) {
        for (int64_t r0 = g; r0 <= more; r0 += G * U) {
          float4 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * G;
            const int64_t at = r == 0 ? 2 * b + 1 : 2 * (b + r);
            v[u] = r <= more ? __ldcg(reinterpret_cast<const float4*>(a.partial + at * a.Hp + c))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            acc.x += v[u].x;
            acc.y += v[u].y;
            acc.z += v[u].z;
            acc.w += v[u].w;
          }
        }
      }
      __syncthreads();
      if (g > 0) sums[g - 1][lane] = acc;
      __syncthreads();
      if (g == 0 && c < a.H) {
#pragma unroll
        for (int q = 0; q < G - 1; ++q) {
          const float4 part = sums[q][lane];
          acc.x += part.x;
          acc.y += part.y;
          acc.z += part.z;
          acc.w += part.w;
        }
        const float v[4] = {acc.x, acc.y, acc.z, acc.w};
        const int64_t at = (int64_t)id * a.lddt + c;
        for (int i = 0; i < 4 && c + i < a.H; ++i)
          store_elem<O>(a.dtable, at + i, fmaf(a.scale, v[i], a.accumulate ? load_elem<O>(a.dtable, at + i) : 0.f));
      }
    }
  }
}

template <typename K, typename... Args>
static cudaError_t launch_pdl(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <typename D, typename O>
static cudaError_t run_lookup_grad(LookupGradArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.N > 0) {
    const SortPlan plan = sort_plan(a.V);
    const size_t smem = sizeof(int) * ((size_t)(kSortThreads / 32 + 2) * (1 << plan.bits) + kSortThreads / 32);
    static KernelMemo memo;
    if (smem > 48 * 1024) {
      e = memo.allow_smem(lookup_grad_sort_kernel, dev.max_smem_optin - 1024, dev);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortCluster);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSortCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, lookup_grad_sort_kernel, a, plan);
    if (e != cudaSuccess) return e;
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  using T = typename D::T;
  using OT = typename O::T;
  a.clearers = a.mark = 0;
  if (!a.accumulate) {
    // A clearing CTA reads all tokens from L2, at about twice the rate of the
    // rows it spares; below 2 KB a row the marks cost more than the rows.
    const int64_t row_bytes = (int64_t)a.H * (int64_t)sizeof(OT);
    const int64_t reads = (a.V / (dev.sm_count * kClearPerSm) + kClearMaxRange) / kClearMaxRange;
    const int64_t token_bytes = a.N * (a.tok64 ? 8 : 4) * reads;
    a.mark = a.N > 0 && row_bytes >= 2048 && kClearPerSm * dev.sm_count * token_bytes <= a.V * row_bytes / 2;
    const unsigned blocks = (unsigned)std::min<int64_t>(a.V, dev.sm_count * kClearPerSm);
    if (a.N == 0) {
      lookup_grad_clear_kernel<O><<<blocks, kClearThreads, 0, s>>>(a);
      return cudaGetLastError();
    }
    if (a.mark) {
      a.clearers = (int)blocks;
    } else {
      e = launch_pdl(lookup_grad_clear_kernel<O>, dim3(blocks), dim3(kClearThreads), 0, s, a);
      if (e != cudaSuccess) return e;
    }
  }
  const unsigned tiles = (unsigned)((a.N + a.tile - 1) / a.tile);
  // as many threads as a row of 16 (fp32: 8) columns a thread has (all of them
  // where they clear too)
  const int threads = a.mark ? kTileThreads : std::min(kTileThreads, chunk_threads(a.H, 32 / (int)sizeof(T)));
  const int per = threads * 32 / (int)sizeof(T);
  a.col_blocks = std::min((a.H + per - 1) / per, 64);
  const dim3 grid(a.clearers + tiles * a.col_blocks);
  GranuleRule in, out;
  in.add(a.dh, a.lddh, sizeof(T));
  out.add(a.dtable, a.lddt, sizeof(OT));
  const int vec = out.bytes(a.H, sizeof(OT)) >= 16;
  e = in.bytes(a.H, sizeof(T)) >= 16
          ? launch_pdl(lookup_grad_tile_kernel<D, O, 16>, grid, dim3(threads), 0, s, a, vec)
          : launch_pdl(lookup_grad_tile_kernel<D, O, (int)sizeof(T)>, grid, dim3(threads), 0, s, a, vec);
  if (e != cudaSuccess || tiles == 1) return e;
  const dim3 joins(std::min<unsigned>(tiles - 1, 2 * dev.sm_count), (unsigned)std::min((a.H + 255) / 256, 64));
  return launch_pdl(lookup_grad_join_kernel<O>, joins, dim3(kJoinThreads), 0, s, a);
}

template <typename D>
cudaError_t launch_lookup_grad(LookupGradArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  a.err = dev.err;
  a.tile = lookup_tile(a.N);
  if (a.N == 0 && a.accumulate) return cudaSuccess;
  if (a.w_f32) return run_lookup_grad<D, F32>(a, dev, s);
  return run_lookup_grad<D, D>(a, dev, s);
}

}  // namespace normk
