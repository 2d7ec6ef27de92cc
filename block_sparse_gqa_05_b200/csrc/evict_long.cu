// Choosing the rows of an eviction with the whole GPU: long rows.
//
// The same order and the same lists as a cluster makes, found by a few kernels
// one after the other, each CTA with one chunk of kChunk rows: sums over a
// (sequence, group) are integers added up in memory between the kernels, so no
// order of atomics can change the result.
//   first   weights and positions are read once: the histogram of the keys' high
//           digit as if no row always stayed, and each chunk's range of positions
//   fixed   chunks whose range holds rows that always stay (few, unless they were
//           asked for) take these out of that histogram into one of their own
//   middle  the histogram of the next digit among the rows at the first; rows above
//           are counted, those at it listed
//   last    the histogram of the last digit, from the lists (or, where one ran
//           over, from the rows)
//   count   what each chunk has above and at the cut, before and past row n, from
//           the same
//   lists   holes and movers at ranks that follow from the chunks before, and
//           what weights and positions show afterwards
// Only chunks with rows that always stay read positions again.  So a row costs 8
// bytes read once, 4 bytes twice from L2, and 8 bytes written.  8 of 1,048,576
// rows with 65,536 to keep: 104 us (slices of a cluster each, read again in every
// pass, 210); each kernel takes some 3 us when there is little to do, the lists 40
// us of the 104.
#include <algorithm>

#include "evict.cuh"

namespace msa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 4;                        // steps of a warp, all loads in flight
constexpr int kChunk = kWarps * kSteps * kStep;  // 8192 rows
constexpr int kCand = 2048;                      // entries of a chunk's list

struct __align__(16) Chunk {
  int pos_min, pos_max;
  int gt_lo, gt_hi, eq_lo, eq_hi;   // above / at the cut, before / past row n
  int cand;                         // rows at the first digit
  int pad;
};

struct State {
  int top;             // largest position
  int fixed;           // rows that always stay
  uint32_t cut[3];     // what is known of the n-th largest key after a digit
  int need[3];         // and its rank among the keys with these digits
};

enum Hist { kHistAll, kHistFixed, kHistMiddle, kHistLast, kHists };

struct LongParams {
  EvictParams p;
  Chunk* chunks;       // [B*G, nch]
  uint32_t* cand;      // [B*G, nch, kCand]
  uint32_t* hist;      // [B*G, kHists, kBins]
  State* states;       // [B*G]
  int nch;
};

// The CTA's chunk.
struct Where {
  int bg, b, c, len, n, x0, x1, y0;
  long long base;
  Chunk* chunk;
  uint32_t* hist;
  State* state;
};

__device__ __forceinline__ Where locate(const LongParams& a) {
  Where o;
  o.bg = static_cast<int>(blockIdx.x) / a.nch;
  o.c = static_cast<int>(blockIdx.x) - o.bg * a.nch;
  o.b = o.bg / a.p.G;
  o.len = min(max(__ldcg(a.p.lens + o.b), 0), a.p.C);
  o.n = min(o.len, a.p.budget);
  o.x0 = static_cast<int>(min(static_cast<long long>(o.len), static_cast<long long>(o.c) * kChunk));
  o.x1 = static_cast<int>(min(static_cast<long long>(o.len), static_cast<long long>(o.x0) + kChunk));
  o.y0 = o.x0 + static_cast<int>(threadIdx.x >> 5) * (kSteps * kStep);
  o.base = static_cast<long long>(o.bg) * a.p.C;
  o.chunk = a.chunks + static_cast<long long>(o.bg) * a.nch + o.c;
  o.hist = a.hist + static_cast<long long>(o.bg) * kHists * kBins;
  o.state = a.states + o.bg;
  return o;
}

__device__ __forceinline__ bool has_fixed(const EvictParams& p, const Chunk* c, int top) {
  const int2 range = __ldcg(reinterpret_cast<const int2*>(&c->pos_min));
  return stays(p, range.x, top) || stays(p, range.y, top);
}

// This lane's rows of the chunk, four a step, from an array of the caller's.
template <bool VEC, typename T>
__device__ __forceinline__ void load_rows(const T* from, const Where& o, T (*v)[4]) {
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int x = o.y0 + u * kStep + 4 * static_cast<int>(threadIdx.x & 31);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[u][e] = T(0);
    if (x < o.x1) load4<VEC>(from + o.base, x, o.x1, v[u]);
  }
}

// Turns the weights of the lane's rows into keys (any value past the chunk).
// ``fixed``: whether rows that always stay are among them, ``only_fixed``:
// whether only these count.
template <bool VEC>
__device__ __forceinline__ void make_keys(const EvictParams& p, const Where& o, bool fixed, bool only_fixed,
                                          int top, const float (*w)[4], uint32_t (*key)[4]) {
#pragma unroll
  for (int u = 0; u < kSteps; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) key[u][e] = weight_key(w[u][e]);
  if (!fixed && !only_fixed) return;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int x = o.y0 + u * kStep + 4 * static_cast<int>(threadIdx.x & 31);
    int q[4] = {0, 0, 0, 0};
    if (fixed && x < o.x1) load4<VEC>(p.pos_in + o.base, x, o.x1, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool f = fixed && stays(p, q[e], top);
      if (f != only_fixed) key[u][e] = f ? kStays : 0u;
    }
  }
}

// The lane's rows before row n, a bit each.
__device__ __forceinline__ uint32_t rows_below(const Where& o, int n) {
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int left = n - (o.y0 + u * kStep + 4 * static_cast<int>(threadIdx.x & 31));
    m |= ((1u << min(max(left, 0), 4)) - 1u) << (4 * u);
  }
  return m;
}

// Counts one bin a lane where in, equal ones (ties) at once.
__device__ __forceinline__ void count_bin(uint32_t* hist, bool in, uint32_t bin) {
  const unsigned m = __ballot_sync(0xffffffffu, in);
  if (!m) return;
  const uint32_t lead = __shfl_sync(0xffffffffu, bin, __ffs(m) - 1);
  if (__all_sync(0xffffffffu, !in || bin == lead)) {
    if ((threadIdx.x & 31) == 0) atomicAdd(hist + lead, static_cast<uint32_t>(__popc(m)));
  } else if (in) {
    atomicAdd(hist + bin, 1u);
  }
}

// Ranks of the warp's rows with a bit in m, in row order: those of a step before
// this lane's, a byte each (at most 128), and the step's number in total.
__device__ __forceinline__ uint32_t rank_rows(uint32_t m, uint32_t* total) {
  uint32_t mine = 0;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) mine |= static_cast<uint32_t>(__popc(m >> (4 * u) & 15u)) << (8 * u);
  uint32_t all = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, all, i);
    if ((threadIdx.x & 31) >= i) all += t;
  }
  *total = __shfl_sync(0xffffffffu, all, 31);
  return all - mine;
}

// Writes the rows with a bit in m, as offsets in the chunk, at their ranks from at.
__device__ __forceinline__ void list_rows(uint32_t m, int y, int at, uint16_t* list) {
  uint32_t total;
  const uint32_t before = rank_rows(m, &total);
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    int r = at + static_cast<int>(before >> (8 * u) & 255u);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m >> (4 * u + e) & 1u) list[r++] = static_cast<uint16_t>(y + u * kStep + e);
    at += static_cast<int>(total >> (8 * u) & 255u);
  }
}

__device__ __forceinline__ void clear_hist(uint32_t* s_hist) {
#pragma unroll
  for (int i = 0; i < kBins / kThreads; ++i) s_hist[threadIdx.x + i * kThreads] = 0;
  __syncthreads();
}

// Finds the bin that holds the need-th largest key; v: the thread's four bins,
// ``more``: what the last bin has besides.  Returns the bin, and the rank in it
// in need.
__device__ __forceinline__ uint4 load_bins(const uint32_t* hist) {
  return __ldcg(reinterpret_cast<const uint4*>(hist) + threadIdx.x);
}
__device__ __forceinline__ uint32_t find_digit(uint4 v, uint32_t more, int* need) {
  __shared__ uint32_t s_sum[kWarps], s_bin;
  __shared__ int s_need;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const uint32_t bins[4] = {v.x, v.y, v.z, v.w + (tid == kThreads - 1 ? more : 0u)};
  const uint32_t mine = bins[0] + bins[1] + bins[2] + bins[3];
  uint32_t above = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const uint32_t t = __shfl_down_sync(0xffffffffu, above, i);
    if (lane + i < 32) above += t;
  }
  if (lane == 0) s_sum[warp] = above;
  __syncthreads();
  above -= mine;
  above += __reduce_add_sync(0xffffffffu, lane > warp && lane < kWarps ? s_sum[lane] : 0u);
  const uint32_t nd = static_cast<uint32_t>(*need);
#pragma unroll
  for (int e = 3; e >= 0; --e) {
    if (above < nd && above + bins[e] >= nd) {
      s_bin = static_cast<uint32_t>(4 * tid + e);
      s_need = static_cast<int>(nd - above);
    }
    above += bins[e];
  }
  __syncthreads();
  *need = s_need;
  return s_bin;
}

// Sums over the CTA of N values a thread; every thread gets them.
template <int N>
__device__ __forceinline__ void sum_cta(int* v) {
  __shared__ int s[kWarps][N];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = __reduce_add_sync(0xffffffffu, v[i]);
    if (lane == 0) s[warp][i] = t;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __reduce_add_sync(0xffffffffu, lane < kWarps ? s[lane][i] : 0);
}

// The histograms and counts of all (sequence, group)s, set to zero.
__global__ void __launch_bounds__(kThreads) evict_zero_kernel(const __grid_constant__ LongParams a) {
  griddep_wait();
  griddep_launch_dependents();
  const long long bg = blockIdx.x;
  uint4* hist = reinterpret_cast<uint4*>(a.hist + bg * kHists * kBins);
#pragma unroll 1
  for (int i = static_cast<int>(threadIdx.x); i < kHists * kBins / 4; i += kThreads)
    hist[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) a.states[bg].fixed = 0;
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 2) evict_first_kernel(const __grid_constant__ LongParams a) {
  __shared__ uint32_t s_hist[kBins];
  __shared__ int s_min[kWarps], s_max[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const Where o = locate(a);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  if (o.c == 0 && tid == 0) {
    const int len = __ldcg(a.p.lens + o.b);
    if (len < 0 || len > a.p.C) atomicOr(a.p.err, kErrBadLength);
    if (o.bg == o.b * a.p.G) a.p.new_lens[o.b] = o.n;
  }
  if (o.n == o.len || o.x0 >= o.x1) return;
  float w[kSteps][4];
  int q[kSteps][4];
  load_rows<VEC>(a.p.w_in, o, w);
  load_rows<VEC>(a.p.pos_in, o, q);
  clear_hist(s_hist);
  int lo = INT32_MAX, hi = INT32_MIN;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int x = o.y0 + u * kStep + 4 * lane;
    bool in[4];
    uint32_t bin[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      in[e] = x + e < o.x1;
      bin[e] = weight_key(w[u][e]) >> 21;
      lo = min(lo, in[e] ? q[u][e] : INT32_MAX);
      hi = max(hi, in[e] ? q[u][e] : INT32_MIN);
    }
    count_bins(s_hist, in, bin);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    s_min[tid >> 5] = lo;
    s_max[tid >> 5] = hi;
  }
  __syncthreads();
  if (tid < 32) {
    lo = __reduce_min_sync(0xffffffffu, lane < kWarps ? s_min[lane] : INT32_MAX);
    hi = __reduce_max_sync(0xffffffffu, lane < kWarps ? s_max[lane] : INT32_MIN);
    if (lane == 0) {
      o.chunk->pos_min = lo;
      o.chunk->pos_max = hi;
    }
  }
#pragma unroll
  for (int i = 0; i < kBins / kThreads; ++i) {
    const int bin = tid + i * kThreads;
    if (s_hist[bin]) atomicAdd(o.hist + kHistAll * kBins + bin, s_hist[bin]);
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 2) evict_fixed_kernel(const __grid_constant__ LongParams a) {
  __shared__ uint32_t s_hist[kBins];
  __shared__ int s_max[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const Where o = locate(a);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  if (o.n == o.len || o.x0 >= o.x1) return;
  const int nch = (o.len - 1) / kChunk + 1;
  int top = INT32_MIN;
#pragma unroll 1
  for (int i = tid; i < nch; i += kThreads) top = max(top, __ldcg(&(o.chunk - o.c + i)->pos_max));
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s_max[tid >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, s_max[lane & (kWarps - 1)]);
  if (o.c == 0 && tid == 0) o.state->top = top;
  if (!has_fixed(a.p, o.chunk, top)) return;
  float w[kSteps][4];
  int q[kSteps][4];
  load_rows<VEC>(a.p.w_in, o, w);
  load_rows<VEC>(a.p.pos_in, o, q);
  clear_hist(s_hist);
  int fixed = 0;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int x = o.y0 + u * kStep + 4 * lane;
    bool in[4];
    uint32_t bin[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      in[e] = x + e < o.x1 && stays(a.p, q[u][e], top);
      bin[e] = weight_key(w[u][e]) >> 21;
      fixed += in[e] ? 1 : 0;
    }
    count_bins(s_hist, in, bin);
  }
  sum_cta<1>(&fixed);
  if (tid == 0) atomicAdd(&o.state->fixed, fixed);
#pragma unroll
  for (int i = 0; i < kBins / kThreads; ++i) {
    const int bin = tid + i * kThreads;
    if (s_hist[bin]) {
      atomicAdd(o.hist + kHistFixed * kBins + bin, s_hist[bin]);
      atomicSub(o.hist + kHistAll * kBins + bin, s_hist[bin]);
    }
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 3) evict_middle_kernel(const __grid_constant__ LongParams a) {
  __shared__ uint32_t s_hist[kBins], s_list[kChunk];
  __shared__ int s_cand;
  griddep_wait();
  griddep_launch_dependents();
  const Where o = locate(a);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  if (o.n == o.len || o.x0 >= o.x1) return;
  // all that has to be read, on its way together
  float w[kSteps][4];
  load_rows<VEC>(a.p.w_in, o, w);
  const uint4 bins = load_bins(o.hist + kHistAll * kBins);
  const uint4 bins_fixed = load_bins(o.hist + kHistFixed * kBins);
  const int top = __ldcg(&o.state->top), n_fixed = __ldcg(&o.state->fixed);
  const bool fixed = has_fixed(a.p, o.chunk, top), only_fixed = n_fixed > o.n;
  if (tid == 0) s_cand = 0;
  clear_hist(s_hist);
  int need = o.n;
  const uint32_t digit = find_digit(only_fixed ? bins_fixed : bins,
                                    only_fixed ? 0u : static_cast<uint32_t>(n_fixed), &need);
  if (o.c == 0 && tid == 0) {
    o.state->cut[0] = digit << 21;
    o.state->need[0] = need;
  }
  uint32_t key[kSteps][4];
  make_keys<VEC>(a.p, o, fixed, only_fixed, top, w, key);
  // rows at the digit or above and those above, a bit each (a row that does not
  // count has key 0, below every digit: a row's key is past 2^21)
  uint32_t ins = 0, gts = 0;
  const uint32_t lo = digit << 21, hi = lo | 0x1fffffu;
#pragma unroll
  for (int u = 0; u < kSteps; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (key[u][e] >= lo) ins |= 1u << (4 * u + e);
      if (key[u][e] > hi) gts |= 1u << (4 * u + e);
    }
  const uint32_t valid = rows_below(o, o.x1);
  gts &= valid;
  ins &= valid & ~gts;
  const uint32_t los = rows_below(o, o.n);
  int gt[2] = {__popc(gts & los), __popc(gts & ~los)};
  // those at the digit: their lower digits and whether they lie before row n, in
  // any order, close together in shared memory first
  {
    const int mine = __popc(ins);
    int at = mine;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, at, i);
      if (lane >= i) at += t;
    }
    int first = 0;
    if (lane == 31 && at) first = atomicAdd(&s_cand, at);
    at += __shfl_sync(0xffffffffu, first, 31) - mine;
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (ins >> (4 * u + e) & 1u)
          s_list[at++] = (key[u][e] & 0x1fffffu) | (los >> (4 * u + e) & 1u ? 0u : 1u << 21);
  }
  sum_cta<2>(gt);
  if (tid == 0) {
    o.chunk->gt_lo = gt[0];
    o.chunk->gt_hi = gt[1];
    o.chunk->cand = s_cand;
  }
  const int listed = s_cand;
  uint32_t* cand = a.cand + (static_cast<long long>(o.bg) * a.nch + o.c) * kCand;
#pragma unroll 1
  for (int i0 = tid - lane; i0 < listed; i0 += kThreads) {
    const bool in = i0 + lane < listed;
    const uint32_t v = in ? s_list[i0 + lane] : 0u;
    count_bin(s_hist, in, v >> 10 & 2047u);
    if (in && i0 + lane < kCand) cand[i0 + lane] = v;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBins / kThreads; ++i) {
    const int bin = tid + i * kThreads;
    if (s_hist[bin]) atomicAdd(o.hist + kHistMiddle * kBins + bin, s_hist[bin]);
  }
}

// Calls f(in, entry) for the chunk's rows at the first digit, in whole warps, from
// its list, or from the rows when it ran over.
template <bool VEC, typename F>
__device__ __forceinline__ void for_cands(const LongParams& a, const Where& o, F f) {
  const int listed = __ldcg(&o.chunk->cand), lane = static_cast<int>(threadIdx.x & 31);
  if (listed <= kCand) {
    const uint32_t* cand = a.cand + (static_cast<long long>(o.bg) * a.nch + o.c) * kCand;
#pragma unroll 1
    for (int i0 = static_cast<int>(threadIdx.x) - lane; i0 < listed; i0 += kThreads) {
      const bool in = i0 + lane < listed;
      f(in, in ? __ldcg(cand + i0 + lane) : 0u);
    }
    return;
  }
  const int top = __ldcg(&o.state->top);
  const uint32_t digit = __ldcg(&o.state->cut[0]) >> 21;
  float w[kSteps][4];
  uint32_t key[kSteps][4];
  load_rows<VEC>(a.p.w_in, o, w);
  make_keys<VEC>(a.p, o, has_fixed(a.p, o.chunk, top), __ldcg(&o.state->fixed) > o.n, top, w, key);
#pragma unroll
  for (int u = 0; u < kSteps; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = o.y0 + u * kStep + 4 * lane + e;
      f(x < o.x1 && key[u][e] >> 21 == digit, (key[u][e] & 0x1fffffu) | (x < o.n ? 0u : 1u << 21));
    }
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 3) evict_last_kernel(const __grid_constant__ LongParams a) {
  __shared__ uint32_t s_hist[kBins];
  griddep_wait();
  griddep_launch_dependents();
  const Where o = locate(a);
  const int tid = static_cast<int>(threadIdx.x);
  if (o.n == o.len || o.x0 >= o.x1) return;
  const uint4 bins = load_bins(o.hist + kHistMiddle * kBins);
  int need = __ldcg(&o.state->need[0]);
  const uint32_t known = __ldcg(&o.state->cut[0]);
  clear_hist(s_hist);
  const uint32_t digit = find_digit(bins, 0u, &need);
  if (o.c == 0 && tid == 0) {
    o.state->cut[1] = known | digit << 10;
    o.state->need[1] = need;
  }
  for_cands<VEC>(a, o, [&](bool in, uint32_t v) {
    count_bin(s_hist, in && (v >> 10 & 2047u) == digit, v & 1023u);
  });
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBins / 2 / kThreads; ++i) {
    const int bin = tid + i * kThreads;
    if (s_hist[bin]) atomicAdd(o.hist + kHistLast * kBins + bin, s_hist[bin]);
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 3) evict_count_kernel(const __grid_constant__ LongParams a) {
  griddep_wait();
  griddep_launch_dependents();
  const Where o = locate(a);
  const int tid = static_cast<int>(threadIdx.x);
  if (o.n == o.len || o.x0 >= o.x1) return;
  const uint4 bins = load_bins(o.hist + kHistLast * kBins);
  int need = __ldcg(&o.state->need[1]);
  const uint32_t cut = __ldcg(&o.state->cut[1]) | find_digit(bins, 0u, &need);
  if (o.c == 0 && tid == 0) {
    o.state->cut[2] = cut;
    o.state->need[2] = need;
  }
  int c4[4] = {0, 0, 0, 0};      // gt_lo, gt_hi, eq_lo, eq_hi among the rows at the first digit
  for_cands<VEC>(a, o, [&](bool in, uint32_t v) {
    const uint32_t low = v & 0x1fffffu, at = cut & 0x1fffffu;
    const bool hi = v >> 21;
    c4[0] += in && low > at && !hi ? 1 : 0;
    c4[1] += in && low > at && hi ? 1 : 0;
    c4[2] += in && low == at && !hi ? 1 : 0;
    c4[3] += in && low == at && hi ? 1 : 0;
  });
  sum_cta<4>(c4);
  if (tid == 0) {
    o.chunk->gt_lo = __ldcg(&o.chunk->gt_lo) + c4[0];
    o.chunk->gt_hi = __ldcg(&o.chunk->gt_hi) + c4[1];
    o.chunk->eq_lo = c4[2];
    o.chunk->eq_hi = c4[3];
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 3) evict_lists_kernel(const __grid_constant__ LongParams a) {
  __shared__ int s_warp[kWarps][4];
  __shared__ uint16_t s_hole[kChunk], s_move[kChunk];
  griddep_wait();
  griddep_launch_dependents();
  const Where o = locate(a);
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const EvictParams& p = a.p;
  if (o.n == o.len) {
    if (o.c == 0 && tid == 0) p.n_moves[o.bg] = 0;
    const bool same_w = p.w_out == p.w_in, same_p = p.pos_out == p.pos_in;
#pragma unroll 1
    for (int x = o.x0 + tid; x < o.x1; x += kThreads) {
      if (!same_w) p.w_out[o.base + x] = __ldcg(p.w_in + o.base + x);
      if (!same_p) p.pos_out[o.base + x] = __ldcg(p.pos_in + o.base + x);
    }
    return;
  }
  if (o.x0 >= o.x1) return;
  const uint32_t cut = __ldcg(&o.state->cut[2]);
  const int need = __ldcg(&o.state->need[2]);    // rows at the cut that stay, the lowest ones
  uint32_t gts = 0, eqs = 0;                     // rows above and at the cut, a bit each
  {
    float w[kSteps][4];
    uint32_t key[kSteps][4];
    load_rows<VEC>(p.w_in, o, w);
    const int top = __ldcg(&o.state->top);
    make_keys<VEC>(p, o, has_fixed(p, o.chunk, top), __ldcg(&o.state->fixed) > o.n, top, w, key);
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (key[u][e] > cut) gts |= 1u << (4 * u + e);
        if (key[u][e] == cut) eqs |= 1u << (4 * u + e);
      }
  }
  const uint32_t los = rows_below(o, o.n), ins = rows_below(o, o.x1);
  gts &= ins;
  eqs &= ins;
  // what comes before this chunk, and all rows at the cut and past row n
  int sum[7] = {0, 0, 0, 0, 0, 0, 0};
  const int nch = (o.len - 1) / kChunk + 1;
#pragma unroll 1
  for (int i = tid; i < nch; i += kThreads) {
    const Chunk* c = o.chunk - o.c + i;
    const int v[4] = {__ldcg(&c->gt_lo), __ldcg(&c->gt_hi), __ldcg(&c->eq_lo), __ldcg(&c->eq_hi)};
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += i < o.c ? v[e] : 0;
    sum[4] += v[2];
    sum[5] += v[1];
    sum[6] += v[3];
  }
  sum_cta<7>(sum);
  // the rows at the cut before row n come before those past it
  const int need_hi = max(need - sum[4], 0);
  if (o.c == 0 && tid == 0) p.n_moves[o.bg] = sum[5] + min(need_hi, sum[6]);
  int c4[4] = {__popc(gts & los), __popc(gts & ~los), __popc(eqs & los), __popc(eqs & ~los)};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c4[e] = __reduce_add_sync(0xffffffffu, c4[e]);
    if (lane == 0) s_warp[warp][e] = c4[e];
  }
  __syncthreads();
  // before this warp, and in the chunk
  int in_warps[4], in_chunk[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int v = lane < kWarps ? s_warp[lane][e] : 0;
    in_warps[e] = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
    in_chunk[e] = __reduce_add_sync(0xffffffffu, v);
  }
  auto holes_before = [&](int x, int gt, int eq) { return min(x, o.n) - gt - min(need, eq); };
  auto moves_before = [&](int gt, int eq) { return gt + min(need_hi, eq); };
  const int hole0 = holes_before(o.x0, sum[0], sum[2]), move0 = moves_before(sum[1], sum[3]);
  const int n_holes = holes_before(o.x1, sum[0] + in_chunk[0], sum[2] + in_chunk[2]) - hole0;
  const int n_moves = moves_before(sum[1] + in_chunk[1], sum[3] + in_chunk[3]) - move0;
  uint32_t keeps = gts;
  if (in_chunk[2] + in_chunk[3]) {
    uint32_t total;
    const uint32_t before = rank_rows(eqs, &total);
    int at = sum[2] + sum[3] + in_warps[2] + in_warps[3];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      int r = at + static_cast<int>(before >> (8 * u) & 255u);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (eqs >> (4 * u + e) & 1u) keeps |= (r++ < need ? 1u : 0u) << (4 * u + e);
      at += static_cast<int>(total >> (8 * u) & 255u);
    }
  }
  const int y = o.y0 - o.x0 + 4 * lane;
  if (n_holes)
    list_rows(ins & los & ~keeps, y,
              holes_before(min(o.y0, o.x1), sum[0] + in_warps[0], sum[2] + in_warps[2]) - hole0, s_hole);
  if (n_moves)
    list_rows(keeps & ~los, y, moves_before(sum[1] + in_warps[1], sum[3] + in_warps[3]) - move0, s_move);
  __syncthreads();
  int32_t* holes = p.holes + static_cast<long long>(o.bg) * p.half + hole0;
  Mover* movers = p.movers + static_cast<long long>(o.bg) * p.half + move0;
  const float* wi = p.w_in + o.base;
  const int32_t* pos = p.pos_in + o.base;
#pragma unroll 1
  for (int i = tid; i < n_holes; i += kThreads) holes[i] = o.x0 + s_hole[i];
#pragma unroll 2
  for (int i = tid; i < n_moves; i += kThreads) {
    const int x = o.x0 + s_move[i];
    movers[i] = Mover{x, __ldcg(wi + x), __ldcg(pos + x), 0};
  }
  __syncthreads();                     // read before they are overwritten
  // what the rows show afterwards: those before row n what they had (a hole gets
  // its mover's with the row), the others nothing
  float* wo = p.w_out + o.base;
  int32_t* po = p.pos_out + o.base;
  const int x_n = min(max(o.x0, o.n), o.x1);
  if (wo != wi || po != pos) {
#pragma unroll 2
    for (int x = o.x0 + tid; x < x_n; x += kThreads) {
      wo[x] = __ldcg(wi + x);
      po[x] = __ldcg(pos + x);
    }
  }
  const int x_v = VEC ? min((x_n + 3) & ~3, o.x1) : o.x1, x_e = VEC ? max(x_v, o.x1 & ~3) : o.x1;
#pragma unroll 1
  for (int x = x_v + 4 * tid; x < x_e; x += 4 * kThreads) {
    *reinterpret_cast<float4*>(wo + x) = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<int4*>(po + x) = make_int4(-1, -1, -1, -1);
  }
#pragma unroll 1
  for (int x = x_n + tid; x < x_v; x += kThreads) {
    wo[x] = 0.f;
    po[x] = -1;
  }
#pragma unroll 1
  for (int x = x_e + tid; x < o.x1; x += kThreads) {
    wo[x] = 0.f;
    po[x] = -1;
  }
}

struct LongWs {
  size_t chunks, cand, hist, states, bytes;
};

int64_t chunks_of(int64_t C) { return ceil_div(C, kChunk); }

LongWs long_layout(int64_t bg, int64_t C) {
  const size_t rows = static_cast<size_t>(bg), all = rows * static_cast<size_t>(chunks_of(C));
  LongWs w{};
  w.chunks = 0;
  w.cand = w.chunks + align_up(all * sizeof(Chunk), 256);
  w.hist = w.cand + align_up(all * kCand * sizeof(uint32_t), 256);
  w.states = w.hist + rows * kHists * kBins * sizeof(uint32_t);
  w.bytes = w.states + align_up(rows * sizeof(State), 256);
  return w;
}

}  // namespace

size_t evict_long_bytes(int64_t bg, int64_t C) { return long_layout(bg, C).bytes; }

cudaError_t launch_evict_long(const EvictParams& p, int64_t bg, bool vec, void* ws, cudaStream_t st) {
  const LongWs w = long_layout(bg, p.C);
  char* mem = static_cast<char*>(ws);
  LongParams a{};
  a.p = p;
  a.chunks = reinterpret_cast<Chunk*>(mem + w.chunks);
  a.cand = reinterpret_cast<uint32_t*>(mem + w.cand);
  a.hist = reinterpret_cast<uint32_t*>(mem + w.hist);
  a.states = reinterpret_cast<State*>(mem + w.states);
  a.nch = static_cast<int>(chunks_of(p.C));
  const dim3 grid(static_cast<unsigned>(bg * a.nch)), block(kThreads);
  using Kernel = void (*)(LongParams);
  const Kernel kernels[] = {
      vec ? evict_first_kernel<true> : evict_first_kernel<false>,
      vec ? evict_fixed_kernel<true> : evict_fixed_kernel<false>,
      vec ? evict_middle_kernel<true> : evict_middle_kernel<false>,
      vec ? evict_last_kernel<true> : evict_last_kernel<false>,
      vec ? evict_count_kernel<true> : evict_count_kernel<false>,
      vec ? evict_lists_kernel<true> : evict_lists_kernel<false>};
  static const char* const names[] = {"cache_evict_first", "cache_evict_fixed", "cache_evict_middle",
                                      "cache_evict_last", "cache_evict_count", "cache_evict_lists"};
  cudaError_t e;
  {
    ProfScope ps_("cache_evict_zero", st);
    e = launch_dependent(evict_zero_kernel, dim3(static_cast<unsigned>(bg)), block, 0, st, a);
  }
  for (int i = 0; i < 6 && e == cudaSuccess; ++i) {
    ProfScope ps_(names[i], st);
    e = launch_dependent(kernels[i], grid, block, 0, st, a);
  }
  return e;
}

}  // namespace msa
