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

template <typename D>
cudaError_t launch_lookup(LookupArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  a.err = dev.err;
  const int64_t blocks = std::min<int64_t>(a.N, (int64_t)dev.sm_count * 8);
  lookup_loop_kernel<D><<<(unsigned)blocks, kLookupLoopThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// The table's gradient.
//
// Kernel 1 sorts the tokens by id, stably, on one cluster of eight CTAs, while
// the grid's other clusters clear the table's gradient (not when it
// accumulates).  Kernel 2 takes the sorted tokens in tiles of 32: a tile sums
// the gradient rows of each id in it, in position order, and stores the ids
// whose tokens all lie in the tile; the first and the last id of a tile may
// have tokens in its neighbours, and leave one partial row each.  Kernel 3 sums
// the partial rows of those ids in tile order.  Every sum therefore has one
// order, whatever runs first: the gradient is the same bits at every call.
// ---------------------------------------------------------------------------

// Sort: a least-significant-digit radix sort of (id, position) pairs, ids
// 0..V with V for ignored tokens, `bits` a digit.  The cluster's 256 warps own
// equal contiguous parts of the input; a pass counts each warp's digits in
// shared memory, adds the counts up over warps and (through distributed shared
// memory) CTAs into each warp's first place for each digit, and moves the
// pairs in order, lanes of a digit ranked by a match across the warp.  No
// atomics, so equal ids keep their order.
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
    for (int b = lane; b < bins; b += 32) mine[b] = 0;
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const bool on = i0 + lane < hi;
      const unsigned act = __ballot_sync(0xffffffffu, on);
      if (on) {
        const int d = (int)((fetch(i0 + lane).x >> shift) & (unsigned)(bins - 1));
        const unsigned same = __match_any_sync(act, d);
        if ((same & below) == 0) mine[d] += __popc(same);
      }
      __syncwarp();
    }
    __syncthreads();
    // per bin: exclusive prefix over this CTA's warps, and its total
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
      int sum = 0;
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
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const bool on = i0 + lane < hi;
      const unsigned act = __ballot_sync(0xffffffffu, on);
      int d = 0;
      unsigned same = 0u;
      if (on) {
        const uint2 kv = fetch(i0 + lane);
        d = (int)((kv.x >> shift) & (unsigned)(bins - 1));
        same = __match_any_sync(act, d);
        dst[base[d] + mine[d] + __popc(same & below)] = kv;
      }
      __syncwarp();  // every lane has read its counter
      if (on && (same & below) == 0) mine[d] += __popc(same);
      __syncwarp();
    }
    src = dst;
    cluster_sync_all();  // the pass's pairs are visible, its totals read
  }
}

// Kernel 1: cluster 0 sorts, the others clear rows [0, V) of the gradient.
template <typename D, bool F32OUT>
__global__ void __launch_bounds__(kSortThreads) lookup_grad_sort_kernel(const LookupGradArgs a, const SortPlan plan) {
  extern __shared__ __align__(16) int smem_sort[];
  if (blockIdx.x < kSortCluster) {
    sort_tokens(a, plan, smem_sort);
    return;
  }
  using T = typename std::conditional<F32OUT, float, typename D::T>::type;
  const int64_t cta = blockIdx.x - kSortCluster, n = gridDim.x - kSortCluster;
  T* out = reinterpret_cast<T*>(a.dtable);
  const size_t row_bytes = (size_t)a.H * sizeof(T);
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && (a.lddt * sizeof(T)) % 16 == 0 && row_bytes % 16 == 0;
  if (vec && a.lddt == a.H) {
    const int64_t words = a.V * (int64_t)(row_bytes / 16);
    for (int64_t i = cta * kSortThreads + threadIdx.x; i < words; i += n * kSortThreads)
      st_vec(reinterpret_cast<uint4*>(out) + i, make_uint4(0u, 0u, 0u, 0u));
    return;
  }
  for (int64_t v = cta; v < a.V; v += n) {
    T* row = out + v * a.lddt;
    if (vec) {
      for (int i = threadIdx.x; i < (int)(row_bytes / 16); i += kSortThreads)
        st_vec(reinterpret_cast<uint4*>(row) + i, make_uint4(0u, 0u, 0u, 0u));
    } else {
      for (int j = threadIdx.x; j < a.H; j += kSortThreads) row[j] = T(0.f);
    }
  }
}

// Kernel 2: one tile of sorted tokens (blockIdx.x) and 256 columns (blockIdx.y).
template <typename D, bool F32OUT>
__global__ void __launch_bounds__(256) lookup_grad_tile_kernel(const LookupGradArgs a) {
  using T = typename D::T;
  using O = typename std::conditional<F32OUT, F32, D>::type;
  pdl_wait_primary();
  __shared__ uint2 kv[kLookupTile + 2];  // with the neighbours' nearest ids
  const int64_t first = (int64_t)blockIdx.x * kLookupTile;
  const int n = (int)min((int64_t)kLookupTile, a.N - first);
  const unsigned none = 0xffffffffu;  // no id (ids are at most V < 2^31)
  for (int i = threadIdx.x; i < n + 2; i += blockDim.x) {
    const int64_t at = first + i - 1;
    kv[i] = at >= 0 && at < a.N ? __ldcg(a.sorted + at) : make_uint2(none, 0u);
  }
  __syncthreads();
  const int j = blockIdx.y * 256 + threadIdx.x;
  if (j >= a.H) return;
  float sum = 0.f;
  for (int i = 0; i < n; ++i) {
    const unsigned id = kv[i + 1].x;
    if (id == (unsigned)a.V) break;  // ignored tokens sort last
    sum += load_elem<D>(reinterpret_cast<const T*>(a.dh) + (int64_t)kv[i + 1].y * a.lddh, j);
    if (i + 1 < n && kv[i + 2].x == id) continue;  // its last token in the tile
    const bool open_front = kv[0].x == kv[1].x && id == kv[1].x;
    const bool open_back = i + 1 == n && kv[n + 1].x == id;
    if (open_front) {
      a.partial[(size_t)2 * blockIdx.x * a.Hp + j] = sum;
    } else if (open_back) {
      a.partial[((size_t)2 * blockIdx.x + 1) * a.Hp + j] = sum;
    } else {
      const int64_t at = (int64_t)id * a.lddt + j;
      const float old = a.accumulate ? load_elem<O>(a.dtable, at) : 0.f;
      store_elem<O>(a.dtable, at, fmaf(a.scale, sum, old));
    }
    sum = 0.f;
  }
}

// Kernel 3: the ids whose tokens cross tiles; blockIdx.x is the tile boundary.
template <typename D, bool F32OUT>
__global__ void __launch_bounds__(256) lookup_grad_join_kernel(const LookupGradArgs a) {
  using O = typename std::conditional<F32OUT, F32, D>::type;
  pdl_wait_primary();
  const int64_t b = blockIdx.x;
  const int64_t end = (b + 1) * kLookupTile;  // first token of tile b + 1
  const unsigned id = __ldcg(a.sorted + end).x;
  if (id == (unsigned)a.V || __ldcg(a.sorted + end - 1).x != id) return;  // nothing crosses here
  if (b > 0 && __ldcg(a.sorted + b * kLookupTile - 1).x == id) return;    // an earlier boundary has it
  const int j = blockIdx.y * 256 + threadIdx.x;
  if (j >= a.H) return;
  float sum = a.partial[((size_t)2 * b + 1) * a.Hp + j];
  for (int64_t t = b + 1; t * kLookupTile < a.N && __ldcg(a.sorted + t * kLookupTile).x == id; ++t)
    sum += a.partial[(size_t)2 * t * a.Hp + j];
  const int64_t at = (int64_t)id * a.lddt + j;
  const float old = a.accumulate ? load_elem<O>(a.dtable, at) : 0.f;
  store_elem<O>(a.dtable, at, fmaf(a.scale, sum, old));
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

template <typename D, bool F32OUT>
static cudaError_t run_lookup_grad(const LookupGradArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const SortPlan plan = sort_plan(a.V);
  auto kern = lookup_grad_sort_kernel<D, F32OUT>;
  const size_t smem = sizeof(int) * ((size_t)(kSortThreads / 32 + 2) * (1 << plan.bits) + kSortThreads / 32);
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  // one cluster sorts; as many again as the GPU holds clear the gradient
  const int clusters = a.accumulate ? 1 : std::max(2, dev.sm_count / kSortCluster);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * kSortCluster));
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, plan);
  if (e != cudaSuccess) return e;
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.N == 0) return cudaSuccess;
  const unsigned tiles = (unsigned)((a.N + kLookupTile - 1) / kLookupTile);
  const unsigned cols = (unsigned)((a.H + 255) / 256);
  e = launch_pdl(lookup_grad_tile_kernel<D, F32OUT>, dim3(tiles, cols), dim3(256), 0, s, a);
  if (e != cudaSuccess || tiles == 1) return e;
  return launch_pdl(lookup_grad_join_kernel<D, F32OUT>, dim3(tiles - 1, cols), dim3(256), 0, s, a);
}

template <typename D>
cudaError_t launch_lookup_grad(LookupGradArgs a, const DeviceInfo& dev, cudaStream_t s) {
  (void)cudaGetLastError();  // drop a stale, non-sticky error left by an earlier call
  a.err = dev.err;
  if (a.N == 0 && a.accumulate) return cudaSuccess;
  if (a.w_f32) return run_lookup_grad<D, true>(a, dev, s);
  return run_lookup_grad<D, false>(a, dev, s);
}

}  // namespace normk
