// Eviction from the own caches by accumulated attention weight.
//
// Per (sequence, group) the n = min(len, budget) best rows stay, under the
// order (rows that always stay, weight descending, row ascending).  A row gets
// one 32-bit order key (a row that always stays the largest), so the rows to
// keep are those above the n-th largest key and the lowest rows equal to it.
// Kept rows past n then fill, in order, the dropped rows before n: only the
// rows that change places are read and written, which is what the kernel
// costs when a lot is dropped; with little to drop it is bound by reading
// weights and positions, and by latency.
//
// A cluster of CTAs shares one (sequence, group), each with a contiguous slice
// of its rows, whose keys it keeps in shared memory (4 bytes a row, two CTAs an
// SM).  Weights and positions are read once for the keys, as if no row always
// stayed, and each step's range of positions; once the largest position is
// known, the steps whose range holds rows that always stay are corrected (a pass
// for the largest position before that for the keys took 61 against 54 us at 32
// x 128K).  The n-th largest key is found digit by digit (11, 11 and 10 bits)
// from histograms in shared memory that every CTA of the cluster reads over
// distributed shared memory: three passes over the slice whatever the values,
// and no order of atomics can change the result.  Each warp then owns a
// contiguous run of rows, counts, and writes the lists of holes and movers at
// ranks that follow from the counts of the warps and CTAs before it.  A lane
// takes four consecutive rows at a time: with one row a lane a slice was read at
// 16 GB/s an SM.  Rows too long for the cluster's shared memory are chosen by
// kernels of the whole GPU instead (evict_long.cu); the moves are the same.
//
// 256 x 4097 rows with one to drop 14.5 us (2.5 of them at the bandwidth of HBM;
// the rest is a chain of passes with a barrier each); 32 x 100,000 to 131,072
// rows to 32,768: 54 us here and 131 us for the moves (floor of both 125).
#include <cooperative_groups.h>
#include <algorithm>

#include "evict.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = kBins / kThreads;       // bins a thread sums
constexpr int kMaxCluster = 8;
// Most rows of a CTA's slice: as long as two CTAs share an SM.  Past it choosing
// by chunks is faster (160 (sequence, group)s of 49152 rows 265 against 345 us,
// of 32768 185 against 206; 8 of 524288 157 against 212), below it slower (64 of
// 65536 155 against 138 us, one of 32768 34 against 21: seven kernels for one).
constexpr int kMaxSlice = 20480;
// Most rows a CTA moves itself; past it a second kernel moves them with the
// whole GPU (one launch more, against one CTA's share of the bandwidth).
constexpr int kMaxFusedMoves = 128;
// Threads and rows of a CTA of the second kernel: small ones end together (256 and
// 256 192 us with the choice at 32 x 128K rows, 128 and 128 186, 128 and 64 184).
constexpr int kMoveThreads = 128;
constexpr int kMoveRows = 64;

// Moves entries [i0, i1) (no more than s_at holds) of (b, g)'s lists by the CTA: a
// thread per entry finds where the row goes from and to (s_at), then a warp
// takes 32 / (d / 4) rows at a time, 16 bytes of K or V a lane, kMoveDeep of
// them in flight (the addresses found by every lane, with the loads of a row's
// list entry before those of the row, made it wait more than it loaded: 172
// against 137 us for 800 MB; 4 rows in flight 140, more CTAs an SM 147).
constexpr int kMoveDeep = 8;
__device__ __forceinline__ void move_rows(const EvictParams& p, int bg, int i0, int i1,
                                          longlong2* s_at) {
  const int b = bg / p.G, g = bg - b * p.G;
  const int threads = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x);
  const long long list = static_cast<long long>(bg) * p.half, base = static_cast<long long>(bg) * p.C;
#pragma unroll 1
  for (int i = i0 + tid; i < i1; i += threads) {
    const int4 mover = __ldcg(reinterpret_cast<const int4*>(p.movers + list + i));
    const int hole = __ldcg(p.holes + list + i);
    p.w_out[base + hole] = __int_as_float(mover.y);
    p.pos_out[base + hole] = mover.z;
    const long long from = row_at(p, b, g, mover.x), to = row_at(p, b, g, hole);
    s_at[i - i0] = make_longlong2(to < 0 ? -1 : from, to);
  }
  __syncthreads();
  const int lane = tid & 31, per = p.d / 4;    // 16-byte pieces of a row's K and V
  const int at_once = 32 / per, sub = lane / per, piece = lane - sub * per;
  const bool is_v = piece >= per / 2;
  uint16_t* cache = (is_v ? p.v : p.k) + (is_v ? piece - per / 2 : piece) * 8;
  const int rows = i1 - i0, step = threads / 32 * at_once;
#pragma unroll 1
  for (int r0 = (tid >> 5) * at_once + sub; r0 < rows; r0 += step * kMoveDeep) {
    uint4 x[kMoveDeep];
#pragma unroll
    for (int u = 0; u < kMoveDeep; ++u) {
      const int r = r0 + u * step;
      const long long from = r < rows ? s_at[r].x : -1;
      if (from >= 0) x[u] = __ldcs(reinterpret_cast<const uint4*>(cache + from));
    }
#pragma unroll
    for (int u = 0; u < kMoveDeep; ++u) {
      const int r = r0 + u * step;
      if (r < rows && s_at[r].x >= 0) *reinterpret_cast<uint4*>(cache + s_at[r].y) = x[u];
    }
  }
}

// What the CTAs of a cluster tell one another.
struct __align__(16) Shared {
  uint32_t hist[3][kBins];
  uint32_t coarse[3][kBins / 32];   // sums of 32 bins
  int top;                // largest position of the slice
  int fixed;              // rows of the slice that always stay
  int counts[4];          // of the slice: above / at the cut, before / past row n
  int wcounts[kWarps][4]; // of its warps
  uint32_t digit;
  int need;
  int red[kWarps];
  int2 range[kMaxSlice / kStep];    // smallest and largest position of a step
};

// VEC: every row of four starts on a 16-byte boundary in all arrays.
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const __grid_constant__ EvictParams p) {
  __shared__ Shared sh;
  extern __shared__ __align__(16) uint32_t s_key[];
  cg::cluster_group cl = cg::this_cluster();
  const int cs = p.cluster, rank = cs > 1 ? static_cast<int>(cl.block_rank()) : 0;
  const int bg = static_cast<int>(blockIdx.x) / cs, b = bg / p.G, g = bg - b * p.G;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto sync_all = [&] {
    if (cs > 1)
      cl.sync();
    else
      __syncthreads();
  };
  auto of_rank = [&](int r) { return cs > 1 ? cl.map_shared_rank(&sh, r) : &sh; };
#pragma unroll 1
  for (int i = tid; i < 3 * kBins / 4; i += kThreads)
    reinterpret_cast<uint4*>(&sh.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) sh.red[0] = __ldcg(p.lens + b);    // by one thread: it is a hot line of L2
  __syncthreads();                                 // and the histograms are clear
  int len = sh.red[0];
  if (len < 0 || len > p.C) {
    if (tid == 0 && rank == 0) atomicOr(p.err, kErrBadLength);
    len = len < 0 ? 0 : p.C;
  }
  const int n = min(len, p.budget);
  if (rank == 0 && tid == 0) {
    if (g == 0) p.new_lens[b] = n;
    if (n == len) p.n_moves[bg] = 0;
  }
  const long long base = static_cast<long long>(bg) * p.C;
  const float* w = p.w_in + base;
  const int32_t* pos = p.pos_in + base;
  float* wo = p.w_out + base;
  int32_t* po = p.pos_out + base;
  // this CTA's slice [x0, x1), and each warp's run [y0, y1) of it, in whole steps
  const int slice = ((len + cs - 1) / cs + kStep - 1) / kStep * kStep;
  const int x0 = min(len, rank * slice), x1 = min(len, x0 + slice);
  const bool same_w = wo == w, same_p = po == pos;
  if (n == len) {
#pragma unroll 1
    for (int x = x0 + tid; x < x1; x += kThreads) {
      if (!same_w) wo[x] = __ldcg(w + x);
      if (!same_p) po[x] = __ldcg(pos + x);
    }
    return;
  }
  const int run = (slice / kStep + kWarps - 1) / kWarps * kStep;
  const int y0 = min(x1, x0 + warp * run), y1 = min(x1, y0 + run);

  // Keys as if no row always stayed, their first digit's histogram, and the range
  // of positions of each step; short slices keep what was read.
  float* s_w = reinterpret_cast<float*>(s_key + slice);
  int* s_pos = reinterpret_cast<int*>(s_key + 2 * slice);
  int top = INT32_MIN;
#pragma unroll 1
  for (int xb = y0; xb < y1; xb += 2 * kStep) {
    int q[2][4];
    float wx[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = xb + u * kStep + 4 * lane;
      if (x < y1) {
        load4<VEC>(pos, x, y1, q[u]);
        load4<VEC>(w, x, y1, wx[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = xb + u * kStep + 4 * lane;
      if (xb + u * kStep >= y1) break;             // the warp's own bound: uniform
      bool in[4];
      uint32_t key[4], bin[4];
      int least = INT32_MAX, most = INT32_MIN;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        in[e] = x + e < y1;
        key[e] = in[e] ? weight_key(wx[u][e]) : 0u;
        bin[e] = key[e] >> 21;
        least = min(least, in[e] ? q[u][e] : INT32_MAX);
        most = max(most, in[e] ? q[u][e] : INT32_MIN);
      }
      if (x < y1) {
        *reinterpret_cast<uint4*>(s_key + x - x0) = *reinterpret_cast<const uint4*>(key);
        if (p.keep) {
          *reinterpret_cast<float4*>(s_w + x - x0) = *reinterpret_cast<const float4*>(wx[u]);
          *reinterpret_cast<int4*>(s_pos + x - x0) = *reinterpret_cast<const int4*>(q[u]);
        }
      }
      count_bins(sh.hist[0], in, bin);
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
      top = max(top, most);
      if (lane == 0) sh.range[(xb - x0) / kStep + u] = make_int2(least, most);
    }
  }
  if (lane == 0) sh.wcounts[warp][0] = top;
  __syncthreads();
  if (warp == 0) {
    top = __reduce_max_sync(0xffffffffu, lane < kWarps ? sh.wcounts[lane][0] : INT32_MIN);
    if (lane == 0) sh.top = top;
  }
  sync_all();
  top = INT32_MIN;
#pragma unroll 1
  for (int r = 0; r < cs; ++r) top = max(top, of_rank(r)->top);

  // Calls f(x, keys, positions, weights) for every step of this warp's rows, the
  // last two only with ``values``.
  auto for_rows = [&](bool values, auto f) {
#pragma unroll 1
    for (int xb = y0; xb < y1; xb += kStep) {
      const int x = xb + 4 * lane;
      uint32_t key[4] = {0, 0, 0, 0};
      int q[4] = {0, 0, 0, 0};
      float wx[4] = {0.f, 0.f, 0.f, 0.f};
      if (x < y1) {
        *reinterpret_cast<uint4*>(key) = *reinterpret_cast<const uint4*>(s_key + x - x0);
        if (values && p.keep) {
          *reinterpret_cast<float4*>(wx) = *reinterpret_cast<const float4*>(s_w + x - x0);
          *reinterpret_cast<int4*>(q) = *reinterpret_cast<const int4*>(s_pos + x - x0);
        } else if (values) {
          load4<VEC>(w, x, y1, wx);
          load4<VEC>(pos, x, y1, q);
        }
      }
      f(x, key, q, wx);
    }
  };
  // Makes the histogram's sums of 32 bins and lets the cluster see both.
  auto show_hist = [&](int h) {
    __syncthreads();
    const uint4 v = *reinterpret_cast<const uint4*>(&sh.hist[h][tid * kPer]);
    uint32_t c = v.x + v.y + v.z + v.w;
#pragma unroll
    for (int o = 1; o < 32 / kPer; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if ((lane & (32 / kPer - 1)) == 0) sh.coarse[h][tid / (32 / kPer)] = c;
    sync_all();
  };
  // Finds the bin that holds the need-th largest key over the cluster, first
  // among the sums of 32 bins and then in one of them; leaves it in sh.digit and
  // the rank in it in sh.need.  One warp: a few remote loads of each CTA.
  auto find_digit = [&](int h, int need) {
    if (warp == 0) {
      uint32_t c0 = 0, c1 = 0;
#pragma unroll 4
      for (int r = 0; r < cs; ++r) {
        const uint2 v = *reinterpret_cast<const uint2*>(&of_rank(r)->coarse[h][2 * lane]);
        c0 += v.x;
        c1 += v.y;
      }
      // keys in higher groups: an exclusive scan from the top
      auto above_of = [&](uint32_t mine) {
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_down_sync(0xffffffffu, inc, o);
          if (lane + o < 32) inc += v;
        }
        return inc - mine;
      };
      const uint32_t nd = static_cast<uint32_t>(need);
      uint32_t above = above_of(c0 + c1);
      const bool in1 = above < nd && above + c1 >= nd;
      const bool in0 = above + c1 < nd && above + c1 + c0 >= nd;
      const unsigned who = __ballot_sync(0xffffffffu, in0 || in1);
      const int src = __ffs(who) - 1;
      const int group = __shfl_sync(0xffffffffu, 2 * lane + (in1 ? 1 : 0), src);
      const uint32_t before = __shfl_sync(0xffffffffu, in1 ? above : above + c1, src);
      uint32_t c = 0;
#pragma unroll 4
      for (int r = 0; r < cs; ++r) c += of_rank(r)->hist[h][32 * group + lane];
      above = before + above_of(c);
      if (above < nd && above + c >= nd) {
        sh.digit = static_cast<uint32_t>(32 * group + lane);
        sh.need = need - static_cast<int>(above);
      }
    }
    __syncthreads();
  };

  // Rows that always stay come before all others: their keys become the largest,
  // in the steps whose range holds such rows.
  int fixed = 0;
#pragma unroll 1
  for (int xb = y0; xb < y1; xb += kStep) {
    const int2 range = sh.range[(xb - x0) / kStep];
    if (!stays(p, range.x, top) && !stays(p, range.y, top)) continue;
    const int x = xb + 4 * lane;
    if (x >= y1) continue;
    int q[4];
    if (p.keep)
      *reinterpret_cast<int4*>(q) = *reinterpret_cast<const int4*>(s_pos + x - x0);
    else
      load4<VEC>(pos, x, y1, q);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (x + e < y1 && stays(p, q[e], top)) {
        atomicSub(&sh.hist[0][s_key[x + e - x0] >> 21], 1u);
        s_key[x + e - x0] = kStays;
        ++fixed;
      }
  }
  fixed = __reduce_add_sync(0xffffffffu, fixed);
  if (lane == 0) {
    sh.red[warp] = fixed;
    atomicAdd(&sh.hist[0][kStays >> 21], static_cast<uint32_t>(fixed));
  }
  __syncthreads();
  if (warp == 0) {
    fixed = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.red[lane] : 0);
    if (lane == 0) sh.fixed = fixed;
  }
  show_hist(0);
  fixed = 0;
#pragma unroll 1
  for (int r = 0; r < cs; ++r) fixed += of_rank(r)->fixed;
  if (fixed > n) {                      // more than fit: only they have keys, by weight
    sync_all();                         // every CTA has read the histogram's sums and counts
    for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = 0;
    __syncthreads();
    for_rows(true, [&](int x, uint32_t* key, const int*, const float* wx) {
      bool in[4];
      uint32_t bin[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        in[e] = key[e] == kStays;
        key[e] = in[e] ? weight_key(wx[e]) : 0u;
        bin[e] = key[e] >> 21;
      }
      if (x < y1) *reinterpret_cast<uint4*>(s_key + x - x0) = *reinterpret_cast<const uint4*>(key);
      count_bins(sh.hist[0], in, bin);
    });
    show_hist(0);
  }
  find_digit(0, n);
  uint32_t cut = sh.digit << 21;
  int need = sh.need;
#pragma unroll 1
  for (int d = 1; d < 3; ++d) {        // the other two digits
    const int hi = d == 1 ? 21 : 10, lo = d == 1 ? 10 : 0;
    const uint32_t mask = d == 1 ? 2047u : 1023u;
    for_rows(false, [&](int x, const uint32_t* key, const int*, const float*) {
      bool in[4];
      uint32_t bin[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        in[e] = x + e < y1 && (key[e] >> hi) == (cut >> hi);
        bin[e] = (key[e] >> lo) & mask;
      }
      count_bins(sh.hist[d], in, bin);
    });
    show_hist(d);
    find_digit(d, need);
    cut |= sh.digit << lo;
    need = sh.need;
  }
  // need: rows equal to the cut that stay, the lowest ones

  // rows above and at the cut, before and past row n
  int c4[4] = {0, 0, 0, 0};
  for_rows(false, [&](int x, const uint32_t* key, const int*, const float*) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = x + e < y1;
      const int hi = x + e < n ? 0 : 2;
      const bool gt = in && key[e] > cut, eq = in && key[e] == cut;
      c4[0] += hi == 0 && gt ? 1 : 0;
      c4[1] += hi == 0 && eq ? 1 : 0;
      c4[2] += hi == 2 && gt ? 1 : 0;
      c4[3] += hi == 2 && eq ? 1 : 0;
    }
  });
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c4[e] = __reduce_add_sync(0xffffffffu, c4[e]);
    if (lane == 0) sh.wcounts[warp][e] = c4[e];
  }
  __syncthreads();
  if (tid < 4) {
    int s = 0;
#pragma unroll 1
    for (int i = 0; i < kWarps; ++i) s += sh.wcounts[i][tid];
    sh.counts[tid] = s;
  }
  sync_all();
  // ranks at which this warp's ties, holes and movers begin, and all moves
  int eq_at = 0, hole_at = 0, move_at = 0, moves = 0;
  auto add_run = [&](const int* c, int rows_lo, int& e, int& hl, int& mv) {
    const int lo = min(max(need - e, 0), c[1]), hi = min(max(need - e - c[1], 0), c[3]);
    hl += rows_lo - c[0] - lo;
    mv += c[2] + hi;
    e += c[1] + c[3];
  };
  auto rows_before_n = [&](int a, int z) { return max(0, min(z, n) - min(a, n)); };
  {
    int e = 0, hl = 0, mv = 0;
#pragma unroll 1
    for (int r = 0; r < cs; ++r) {
      if (r == rank) {
        eq_at = e;
        hole_at = hl;
        move_at = mv;
      }
      const int a = min(len, r * slice);
      int c[4];
      const Shared* o = of_rank(r);
      for (int i = 0; i < 4; ++i) c[i] = o->counts[i];
      add_run(c, rows_before_n(a, min(len, a + slice)), e, hl, mv);
    }
    moves = mv;
  }
#pragma unroll 1
  for (int i = 0; i < warp; ++i) {
    const int a = min(x1, x0 + i * run);
    add_run(sh.wcounts[i], rows_before_n(a, min(x1, a + run)), eq_at, hole_at, move_at);
  }
  Mover* movers = p.movers + static_cast<long long>(bg) * p.half;
  int32_t* holes = p.holes + static_cast<long long>(bg) * p.half;
  for_rows(true, [&](int x, const uint32_t* key, int* q, float* wx) {
    bool eq[4], keep[4], hole[4], move[4];
    int count;
#pragma unroll
    for (int e = 0; e < 4; ++e) eq[e] = x + e < y1 && key[e] == cut;
    int re = eq_at + rank4(eq, &count);
    eq_at += count;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = x + e < y1, lo = x + e < n;
      keep[e] = in && (key[e] > cut || (eq[e] && re < need));
      re += eq[e] ? 1 : 0;
      hole[e] = in && lo && !keep[e];
      move[e] = keep[e] && !lo;
    }
    int rh = hole_at + rank4(hole, &count);
    hole_at += count;
    int rm = move_at + rank4(move, &count);
    move_at += count;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (hole[e]) holes[rh++] = x + e;
      if (move[e]) movers[rm++] = Mover{x + e, wx[e], q[e], 0};
    }
    // what the rows show afterwards; a hole gets its mover's with the row
    if (x + 3 < min(n, y1) ? !(same_w && same_p) : x < y1) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (x + e >= n) {
          wx[e] = 0.f;
          q[e] = -1;
        }
      if (VEC && x + 4 <= y1) {
        *reinterpret_cast<float4*>(wo + x) = make_float4(wx[0], wx[1], wx[2], wx[3]);
        *reinterpret_cast<int4*>(po + x) = make_int4(q[0], q[1], q[2], q[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x + e < y1) {
            wo[x + e] = wx[e];
            po[x + e] = q[e];
          }
      }
    }
  });
  if (!p.fused) {
    if (rank == 0 && tid == 0) p.n_moves[bg] = moves;
    if (cs > 1) cl.sync();             // no CTA leaves while another reads its counts
    return;
  }
  __threadfence();
  sync_all();
  // this CTA's share, at most kMaxFusedMoves; the histograms' memory is free now
  const int share = (moves + cs - 1) / cs;
  move_rows(p, bg, min(moves, rank * share), min(moves, (rank + 1) * share),
            reinterpret_cast<longlong2*>(&sh.hist[0][0]));
}

// The moves of all (sequence, group)s, kMoveRows a CTA.
__global__ void __launch_bounds__(kMoveThreads, 8)
    evict_move_kernel(const __grid_constant__ EvictParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int bg = blockIdx.x;
  const int n = __ldcg(p.n_moves + bg);
  __shared__ longlong2 s_at[kMoveRows];
#pragma unroll 1
  for (long long i0 = static_cast<long long>(blockIdx.y) * kMoveRows; i0 < n;
       i0 += static_cast<long long>(gridDim.y) * kMoveRows) {
    move_rows(p, bg, static_cast<int>(i0), static_cast<int>(min(static_cast<long long>(n), i0 + kMoveRows)),
              s_at);
    __syncthreads();
  }
}

size_t lists_half(const msa_shape& s) { return static_cast<size_t>(s.seq_kv) / 2; }

struct EvictWs {
  size_t movers, holes, n_moves, chunks, bytes;
};

// Holes and movers of a (sequence, group): at most min(n, len - n) <= N / 2 each.
EvictWs ws_layout(const msa_shape& s) {
  const size_t bg = static_cast<size_t>(s.batch) * s.n_kv_heads, lists = bg * lists_half(s);
  EvictWs w{};
  w.movers = 0;
  w.holes = align_up(lists * sizeof(Mover), 256);
  w.n_moves = w.holes + align_up(lists * sizeof(int32_t), 256);
  w.chunks = w.n_moves + align_up(bg * sizeof(int32_t), 256);
  // with a cluster of one CTA; a larger one may do without
  w.bytes = w.chunks + (s.seq_kv > kMaxSlice ? evict_long_bytes(static_cast<int64_t>(bg), s.seq_kv) : 0);
  return w;
}

cudaError_t launch_clustered(void (*kernel)(EvictParams), unsigned grid, int cluster,
                             size_t smem, cudaStream_t st, const EvictParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

size_t evict_workspace_bytes(const msa_shape& s) { return ws_layout(s).bytes; }

cudaError_t launch_cache_evict(const msa_shape& s, const EvictArgs& a, void* ws, cudaStream_t st) {
  const DevCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const EvictWs w = ws_layout(s);
  char* mem = static_cast<char*>(ws);
  EvictParams p{};
  p.lens = a.lens;
  p.w_in = a.w_in;
  p.pos_in = a.pos_in;
  p.k = a.k;
  p.v = a.v;
  p.w_out = a.w_out;
  p.pos_out = a.pos_out;
  p.new_lens = a.new_lens;
  p.table = a.pages.table;
  p.num_pages = a.pages.num_pages;
  p.movers = reinterpret_cast<Mover*>(mem + w.movers);
  p.holes = reinterpret_cast<int32_t*>(mem + w.holes);
  p.n_moves = reinterpret_cast<int32_t*>(mem + w.n_moves);
  p.err = ctx->err;
  p.G = s.n_kv_heads;
  p.C = s.seq_kv;
  p.d = s.head_dim;
  p.nb = static_cast<int>(ceil_div(s.seq_kv, 128));
  p.budget = a.budget;
  p.n_first = a.n_first;
  p.n_recent = a.n_recent;
  p.half = static_cast<int>(lists_half(s));
  const int64_t bg = static_cast<int64_t>(s.batch) * s.n_kv_heads;
  const int64_t most = std::min<int64_t>(a.budget, std::max(p.C - a.budget, 0));   // moves there can be
  auto vec16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; };
  const bool vec = p.C % 4 == 0 && vec16(p.w_in) && vec16(p.pos_in) && vec16(p.w_out) && vec16(p.pos_out);
  // CTAs of a cluster: as many as run at once, not below 2048 rows each (8 x 8192
  // rows by 4 CTAs 15.8, by 8 17.8 us; one of 2048 by one 11.4, by two 13.6), two
  // an SM; for a cluster of 8 two an SM only from 4096 rows each (32 x 16384 rows
  // by 4 CTAs 28.6, by 8 36.9 us; 32 x 32768 48.5 and 44).  Clusters of 16 had to
  // wait for one another: seven GPCs take two (16 x 65536 rows 74 us, by 8 51).
  p.cluster = 1;
  while (p.cluster < kMaxCluster && 2 * bg * p.cluster <= 2ll * ctx->num_sms &&
         p.C / (2 * p.cluster) >= 2048 &&
         (p.cluster < 4 || 2 * bg * p.cluster <= ctx->num_sms || p.C / (2 * p.cluster) >= 4096))
    p.cluster *= 2;
  const size_t slice = align_up(static_cast<size_t>(ceil_div(p.C, p.cluster)), kStep);
  cudaError_t e = cudaSuccess;
  if (slice > kMaxSlice) {
    e = launch_evict_long(p, bg, vec, mem + w.chunks, st);
  } else {
    p.fused = most <= static_cast<int64_t>(kMaxFusedMoves) * p.cluster;
    // short slices keep weights and positions too (256 x 4096 rows with one to drop
    // 14.6 against 15.2 us, read three times)
    p.keep = 3 * slice <= kMaxSlice;
    auto kernel = vec ? evict_kernel<true> : evict_kernel<false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSlice * 4);
    if (e != cudaSuccess) return e;
    ProfScope ps_("cache_evict", st);
    e = launch_clustered(kernel, static_cast<unsigned>(bg * p.cluster), p.cluster,
                         slice * (p.keep ? 3 : 1) * sizeof(uint32_t), st, p);
  }
  if (e != cudaSuccess || p.fused || most == 0) return e;
  {
    ProfScope ps_("cache_evict_move", st);
    const int64_t slices = std::min<int64_t>(ceil_div(most, kMoveRows), 65535);   // grid limit
    e = launch_dependent(evict_move_kernel, dim3(static_cast<unsigned>(bg), static_cast<unsigned>(slices)),
                         dim3(kMoveThreads), 0, st, p);
  }
  return e;
}

}  // namespace msa
