// What the two ways to choose the rows of an eviction share: its arguments, the
// order of rows, and steps of a warp over 128 rows, four consecutive ones a lane.
// Lengths, weights and positions are read from L2: the kernel before on the
// stream may still write them when this one starts, after an SM cached the line.
#pragma once
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace msa {

constexpr int kBins = 2048;
constexpr int kStep = 128;                   // rows a warp takes at a time, four a lane

// A moved row: where it came from, and its weight and position.
struct __align__(16) Mover {
  int row;
  float weight;
  int pos;
  int pad;     // one 16-byte access
};

struct EvictParams {
  const int32_t* lens;
  const float* w_in;
  const int32_t* pos_in;
  uint16_t *k, *v;
  float* w_out;
  int32_t* pos_out;
  int32_t* new_lens;
  const int32_t* table;
  Mover* movers;      // [B*G, C/2]
  int32_t* holes;     // [B*G, C/2]
  int32_t* n_moves;   // [B*G]
  uint32_t* err;
  int G, C, d, nb, num_pages, budget, n_first, n_recent, half;
  int cluster, fused, keep;
};

// Order key of a weight: larger weight, larger key; NaN as -infinity, -0 as 0.
// All lie between 0, which stands for no row, and kStays.
constexpr uint32_t kStays = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t weight_key(float w) {
  const int u = __float_as_int(isnan(w) ? -INFINITY : w + 0.f);
  return static_cast<uint32_t>(u ^ (u >> 31 | INT32_MIN));     // negative: all bits flipped, else the sign
}

__device__ __forceinline__ bool stays(const EvictParams& p, int pos, int top) {
  return pos < p.n_first || static_cast<long long>(pos) > static_cast<long long>(top) - p.n_recent;
}

// Element offset of row x of (b, g), or -1 (flagged) when its page is bad.
__device__ __forceinline__ long long row_at(const EvictParams& p, int b, int g, int x) {
  if (!p.table) return ((static_cast<long long>(b) * p.G + g) * p.C + x) * p.d;
  const int pg = __ldg(p.table + static_cast<long long>(b) * p.nb + (x >> 7));
  if (pg < 0 || pg >= p.num_pages) {
    atomicOr(p.err, kErrBadPage);
    return -1;
  }
  return ((static_cast<long long>(pg) * p.G + g) * 128 + (x & 127)) * p.d;
}

// Four consecutive elements from x; of those at or past ``end`` the value is
// whatever is there (the arrays go on to a multiple of four), or 0.
template <bool VEC, typename T>
__device__ __forceinline__ void load4(const T* p, int x, int end, T* v) {
  if constexpr (VEC) {
    const int4 q = __ldcg(reinterpret_cast<const int4*>(p + x));
    const T* t = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = x + e < end ? __ldcg(p + x + e) : T(0);
  }
}

// Counts the bins of four rows a lane where in.  Equal keys (rows that no query
// looked at, ties) would queue up on one bin.
__device__ __forceinline__ void count_bins(uint32_t* hist, const bool* in, const uint32_t* bin) {
  const bool any = in[0] || in[1] || in[2] || in[3];
  const unsigned m = __ballot_sync(0xffffffffu, any);
  if (!m) return;
  const uint32_t own = in[0] ? bin[0] : in[1] ? bin[1] : in[2] ? bin[2] : bin[3];
  const uint32_t lead = __shfl_sync(0xffffffffu, own, __ffs(m) - 1);
  bool same = true;
  int c = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    same &= !in[e] || bin[e] == lead;
    c += in[e] ? 1 : 0;
  }
  if (__all_sync(0xffffffffu, same)) {
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0) atomicAdd(hist + lead, static_cast<uint32_t>(c));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (in[e]) atomicAdd(hist + bin[e], 1u);
  }
}

// Rank of this lane's first row with f among the warp's 128, and their number.
__device__ __forceinline__ int rank4(const bool* f, int* count) {
  const unsigned below = (1u << (threadIdx.x & 31)) - 1u;
  int before = 0, all = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const unsigned m = __ballot_sync(0xffffffffu, f[e]);
    before += __popc(m & below);
    all += __popc(m);
  }
  *count = all;
  return before;
}

// evict_long.cu: chooses the rows with the whole GPU (the lists, the weights and
// positions as the rows show them; not the moves).
size_t evict_long_bytes(int64_t bg, int64_t C);
cudaError_t launch_evict_long(const EvictParams& p, int64_t bg, bool vec, void* ws, cudaStream_t st);

}  // namespace msa
