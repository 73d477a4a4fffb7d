// A thread's share of a row: E columns, as granules of GB bytes.  A warp owns
// 32*E contiguous columns: granule g of lane l holds the GE columns from
// 32*GE*g + GE*l of the warp's, so every access of a warp is contiguous and a
// thread reaches its granules from one pointer at constant offsets.  GB is 32
// where rows are 32-byte aligned (one 256-bit access), 16 where they are
// 16-byte aligned, and one element otherwise: odd widths and shifted rows run
// the same kernels, only with narrower accesses.
#pragma once

#include <atomic>

#include "common.cuh"
#include "launch.h"

namespace normk {

template <typename D, int GB, int E_>
struct Chunk {
  using T = typename D::T;
  static constexpr int ES = (int)sizeof(T);
  static constexpr int E = E_;             // columns a thread
  static constexpr int NP = E / 2;         // fp32 pairs
  static constexpr int NW = E * ES / 4;    // packed words
  static constexpr int GE = GB / ES;       // columns a granule
  static constexpr int NG = E / GE;        // granules
  static_assert(GB == 32 || GB == 16 || GB == ES, "granule");
  static_assert(E % GE == 0 && E % 4 == 0, "whole granules");

  // First column of thread t of a row group, and column of its e-th element
  // from there.
  __device__ static __forceinline__ int base(int t) { return (t >> 5) * (32 * E) + (t & 31) * GE; }
  __device__ static __forceinline__ constexpr int col(int e) { return (e / GE) * (32 * GE) + e % GE; }

  // Load the thread's columns from its first, `p` (those `lim` columns or more
  // behind it lie past the row: zeros), as packed words.
  __device__ static __forceinline__ void load(const T* p, int lim, uint32_t (&w)[NW]) {
    if constexpr (GB == 32) {
      static_assert(NG == 1, "one 256-bit access");
      if (0 < lim) {
        ld_stream32(p, w);
      } else {
#pragma unroll
        for (int k = 0; k < NW; ++k) w[k] = 0u;
      }
    } else if constexpr (GB == 16) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint4 u = col(g * GE) < lim ? ld_stream(p + col(g * GE)) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * g] = u.x;
        w[4 * g + 1] = u.y;
        w[4 * g + 2] = u.z;
        w[4 * g + 3] = u.w;
      }
    } else if constexpr (ES == 4) {
#pragma unroll
      for (int g = 0; g < NG; ++g) w[g] = col(g) < lim ? ldg32(p + col(g)) : 0u;
    } else {
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const uint32_t lo = col(2 * k) < lim ? ldg16(p + col(2 * k)) : 0u;
        const uint32_t hi = col(2 * k + 1) < lim ? ldg16(p + col(2 * k + 1)) : 0u;
        w[k] = __byte_perm(lo, hi, 0x5410);
      }
    }
  }

  __device__ static __forceinline__ void store(T* p, int lim, const uint32_t (&w)[NW]) {
    if constexpr (GB == 32) {
      if (0 < lim) st_vec32(p, w);
    } else if constexpr (GB == 16) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (col(g * GE) < lim) st_vec(p + col(g * GE), make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]));
    } else if constexpr (ES == 4) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (col(g) < lim) reinterpret_cast<uint32_t*>(p)[col(g)] = w[g];
    } else {
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (col(g) < lim) reinterpret_cast<uint16_t*>(p)[col(g)] = (uint16_t)(w[g / 2] >> (16 * (g & 1)));
    }
  }

  // Multiply f by the thread's parameters, p the row's (nullptr: ones); 0 past
  // the row.
  __device__ static __forceinline__ void scale_by_param(const void* p, bool f32, int b, int lim, float (&f)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float v = col(e) < lim ? (p ? load_param<D>(p, b + col(e), f32) : 1.f) : 0.f;
      f[e] *= v;
    }
  }

  __device__ static __forceinline__ uint32_t ldg32(const T* p) {
    uint32_t v;
    asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
  }
  __device__ static __forceinline__ uint32_t ldg16(const T* p) {
    uint32_t v;
    asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
  }
};

// fp32 parameters of a thread in shared memory: NV vectors of E floats, then 4
// floats of padding, so that the 16-byte reads of eight consecutive threads
// fall into distinct banks (the stride is 4 mod 32 words for E = 16 and even
// NV, 20 for the others).
template <int E, int NV>
__host__ __device__ constexpr int param_slot() { return NV * E + 4; }

template <int E>
__device__ __forceinline__ void put_params(float* slot, const float (&f)[E]) {
#pragma unroll
  for (int q = 0; q < E / 4; ++q)
    *reinterpret_cast<float4*>(slot + 4 * q) = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
}

// Shared memory by 32-bit address.
template <int W>
__device__ __forceinline__ void lds_words(uint32_t p, uint32_t* w) {
  static_assert(W == 2 || W == 4, "8 or 16 bytes");
  if constexpr (W == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
  else
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(p));
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(p));
  return v;
}
// Pairs 0 and 1 at p (16-byte aligned).
__device__ __forceinline__ void lds_pairs(uint32_t p, float2 (&v)[2]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0].x), "=f"(v[0].y), "=f"(v[1].x), "=f"(v[1].y) : "r"(p));
}

// Sum four values over a row group of nw <= kSum4Warps warps, as group_sum: the
// warp stage is a reduce-scatter (six shuffles; value k ends in lanes
// 8k..8k+7).  `sh` holds kSum4Floats floats; parity alternates per call.
constexpr int kSum4Warps = 24;
constexpr int kSum4Floats = 2 * 4 * kSum4Warps;
__device__ __forceinline__ void group_sum4(float (&v)[4], float* sh, int nw, int wig, int lane, int bar_id, int parity) {
  const bool hi4 = (lane & 16) != 0;
  float k0 = hi4 ? v[2] : v[0], k1 = hi4 ? v[3] : v[1];
  k0 += __shfl_xor_sync(0xffffffffu, hi4 ? v[0] : v[2], 16);
  k1 += __shfl_xor_sync(0xffffffffu, hi4 ? v[1] : v[3], 16);
  const bool hi3 = (lane & 8) != 0;
  float k = hi3 ? k1 : k0;
  k += __shfl_xor_sync(0xffffffffu, hi3 ? k0 : k1, 8);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) k += __shfl_xor_sync(0xffffffffu, k, off);
  if (nw == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, k, 8 * i);
    return;
  }
  // buf[value][warp]; eight lanes a value then add up the warps' partials
  float* buf = sh + parity * (4 * kSum4Warps) + (lane >> 3) * kSum4Warps;
  if ((lane & 7) == 0) buf[wig] = k;
  named_barrier(bar_id, nw * 32);
  float x = 0.f;
#pragma unroll
  for (int i = 0; i < kSum4Warps / 8; ++i)
    if ((lane & 7) + 8 * i < nw) x += buf[(lane & 7) + 8 * i];
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, x, 8 * i);
}

// Granule that every given row tensor allows: 32, 16 or one element.
struct GranuleRule {
  unsigned long long bits = 0;
  void add(const void* p, int64_t ld, size_t es) {
    bits |= (unsigned long long)reinterpret_cast<uintptr_t>(p) | (unsigned long long)(ld * (int64_t)es);
  }
  int bytes(int H, size_t es) const {
    const unsigned long long b = bits | (unsigned long long)H * es;
    return (b & 31u) == 0 ? 32 : (b & 15u) == 0 ? 16 : (int)es;
  }
};

// Launch configuration of a call's first kernel: clusters of `cl` CTAs, and,
// with `early`, programmatic stream serialization, so that its CTAs come up while
// the kernel before it drains (one after another, 8192x1024 bf16 sandwich_rms
// 18.4 -> 15.9 us a call).  Such a kernel reads and writes no global memory
// before pdl_wait_primary(), after which the kernels before it are through, and
// every CTA passes it, so that a kernel that waits for this one has waited for
// those too.  Not for large persistent grids of clusters: brought up one by one
// in the places that the kernel before leaves, they end up unevenly spread over
// the SMs (8192x5120 bf16 sandwich_rms_grad 89 -> 124 us).
struct FirstLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  FirstLaunch(unsigned threads, size_t smem, cudaStream_t s, int cl) {
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  template <typename K, typename... Args>
  cudaError_t launch(unsigned grid, bool early, K kern, Args... args) {
    cfg.gridDim.x = grid;
    cfg.numAttrs = early ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  FirstLaunch(const FirstLaunch&) = delete;
  FirstLaunch& operator=(const FirstLaunch&) = delete;
};

// What a launcher asks the runtime about its kernel, asked once per device and
// shape: at the sizes where a call is all latency, the questions cost more than
// the launch.  One object per kernel (static in its launcher); plain atomics, so
// that calls of several threads at worst ask twice.
class KernelMemo {
 public:
  // Let the kernel have any dynamic shared memory up to `limit` (the same at
  // every call).
  template <typename K>
  cudaError_t allow_smem(K kern, int limit, const DeviceInfo& dev) {
    if (allowed_[dev.id].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, limit);
    if (e == cudaSuccess) allowed_[dev.id].store(true, std::memory_order_release);
    return e;
  }
  // The CTAs (or, asked through `ask`, clusters) resident at once.
  template <typename F>
  int resident(int threads, size_t smem, const DeviceInfo& dev, F&& ask) {
    const unsigned long long key = ((unsigned long long)smem << 32) | ((unsigned long long)threads << 16);
    const unsigned long long seen = resident_[dev.id].load(std::memory_order_relaxed);
    if (seen != 0 && (seen & ~0xffffull) == key) return (int)(seen & 0xffffull);
    int n = 0;
    if (ask(&n) != cudaSuccess || n < 1) return 1;
    n = n < 0xffff ? n : 0xffff;
    resident_[dev.id].store(key | (unsigned long long)n, std::memory_order_relaxed);
    return n;
  }

 private:
  std::atomic<bool> allowed_[kMaxDevices] = {};
  std::atomic<unsigned long long> resident_[kMaxDevices] = {};
};

// Threads a row of H columns at E columns a thread: whole warps.
inline int chunk_threads(int64_t H, int E) { return (int)((H + 32 * E - 1) / (32 * E) * 32); }

}  // namespace normk
