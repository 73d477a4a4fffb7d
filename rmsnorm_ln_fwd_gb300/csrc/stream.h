// Internal interface of the residual-stream operators: the block join
// (sandwich_rms and its gradient) and the token lookup (embedding_lookup,
// embedding_rms, embedding_grad).  stream_api.cu validates the arguments;
// the functions here pick a kernel configuration and launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.h"

namespace normk {

// Block join forward: h = alpha*res + gate*p, y = rmsnorm(h)*gpre, with
// p = rmsnorm(x)*gpost (post) or x.
struct JoinArgs {
  const void* x;
  int64_t ldx;
  const void* res;
  int64_t ldr;
  const void* gpost;  // may be null (ones)
  const void* gate;   // may be null (ones); gate row of row r is r / run
  int64_t ldg;
  const void* gpre;  // may be null (ones)
  void* y;           // null without the norm after the add
  int64_t ldy;
  void* h;
  int64_t ldh;
  float* rpost;  // may be null
  float* rpre;   // may be null
  int64_t N;
  int64_t run;  // rows that share a gate row (N when there is one or none)
  int H;
  float eps;
  float alpha;
  int post, pre;     // which norms are taken
  int w_f32, g_f32;  // gammas / gate are fp32 (else the row dtype)
  unsigned* err;     // device error word (bounded waits; filled in by the launcher)
};

// Its gradient.  Partial rows (fp32, Hp apart): ws_pre[P] for dgamma_pre,
// ws_post[P] for sums of dh*o_hat (one gate row or none) or of gate*dh*o_hat
// (several), ws_seg[2*U] for the runs a unit of rows holds only in part: slot
// 2u of the run its first row is in, slot 2u + 1 of the run its last row is in.
struct JoinGradArgs {
  const void* dy;  // null without the norm after the add
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const void* h;
  int64_t ldh;
  const float* rpost;  // null without the norm after the block
  const float* rpre;   // null without the norm after the add
  const void* gpost;
  const void* gate;
  int64_t ldg;
  const void* gpre;
  const void* dh_in;  // may be null (zeros) when dy is given
  int64_t lddh;
  void* dx;
  int64_t lddx;
  void* dres;
  int64_t lddres;
  void* dgpost;  // may be null
  void* dgate;   // may be null
  int64_t lddg;
  void* dgpre;  // may be null
  float* ws_pre;
  float* ws_post;
  float* ws_seg;
  int64_t N;
  int64_t run;
  int64_t gate_rows;  // 0 or 1: one coefficient row for all rows
  int H;
  int Hp;
  float alpha;
  int w_f32, g_f32;
  int P, U;  // partial rows; row units (U = P * row groups of a CTA)
  int early;  // a small grid, which lets the kernels behind it come up at once
  unsigned* err;
};

// Token lookup.
struct LookupArgs {
  const void* table;
  int64_t ldt;
  int64_t V;
  const void* tokens;
  int tok64;
  const void* gamma;  // may be null (ones)
  void* y;            // null without the norm
  int64_t ldy;
  void* h;
  int64_t ldh;
  float* rstd;  // may be null
  int64_t N;
  int H;
  float eps;
  float scale;
  int w_f32;
  unsigned* err;
};

// The table's gradient from tokens sorted by id.
struct LookupGradArgs {
  const void* dh;
  int64_t lddh;
  const void* tokens;
  int tok64;
  void* dtable;
  int64_t lddt;
  int64_t V;
  int64_t N;
  int H;
  int Hp;
  float scale;
  int64_t padding;  // ignored id, or -1
  int accumulate;
  int w_f32;  // dtable is fp32 (else the row dtype)
  uint2* sorted;  // (id, position), N of them; V as the id of an ignored token
  uint2* other;   // the sort's second buffer
  float* partial;  // [2 * tiles][Hp]
  int2* owners;    // [1 + tiles]: how many ids cross tiles; (the tile it begins in, id) of each
  // filled in by the launcher:
  int tile;        // sorted tokens a tile
  int mark;        // only the rows that no token names are cleared
  int clearers;    // CTAs that clear rows beside the tiles
  int col_blocks;  // CTAs a tile
  unsigned* err;
};

constexpr int kJoinMaxPartialsPerSm = 3;
// Row groups a CTA of the gradient may have: an upper bound by the width, for
// the workspace (groups of at least one warp for every 512 columns, at most 512
// threads and eight groups a CTA).
inline int join_max_groups(int64_t H) {
  const int64_t warps = (H + 511) / 512;
  return warps >= 16 ? 1 : (int)std::min<int64_t>(8, 16 / warps);
}
// Sorted tokens a tile of the table's gradient: few tokens take short tiles,
// for the sake of their number.
constexpr int kLookupMaxTile = 32;
inline int lookup_tile(int64_t N) { return N <= 4096 ? 8 : N <= 8192 ? 16 : kLookupMaxTile; }
// The most tiles any batch of up to N tokens has: the tiles of N, but from 4096
// tokens on not fewer than the 512 that 4096 (of eight) and 8192 (of 16) have.
inline int64_t lookup_max_tiles(int64_t N) {
  const int64_t tiles = (N + lookup_tile(N) - 1) / lookup_tile(N);
  return N >= 4096 ? std::max<int64_t>(tiles, 512) : tiles;
}

// Device error bit of a token id outside the table.
constexpr unsigned kErrBadToken = 4u;

template <typename D>
cudaError_t launch_join(JoinArgs a, const DeviceInfo& dev, cudaStream_t s);
template <typename D>
cudaError_t launch_join_grad(JoinGradArgs a, const DeviceInfo& dev, cudaStream_t s);
template <typename D>
cudaError_t launch_lookup(LookupArgs a, const DeviceInfo& dev, cudaStream_t s);
template <typename D>
cudaError_t launch_lookup_grad(LookupGradArgs a, const DeviceInfo& dev, cudaStream_t s);

}  // namespace normk
