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
// of its rows in shared memory when they fit.  The n-th largest key is found
// digit by digit (11, 11 and 10 bits) from histograms in shared memory that
// every CTA of the cluster reads over distributed shared memory: three passes
// over the slice whatever the values, no order of atomics can change the
// result.  Each warp then owns a contiguous run of rows, counts, and writes
// the lists of holes and movers at ranks that follow from the counts of the
// warps and CTAs before it.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kPer = kBins / kThreads;       // bins a thread sums
constexpr int kMaxCluster = 8;
// Most rows a CTA keeps in shared memory (position and key, 8 bytes each).
constexpr int kMaxStash = 24576;
// Most rows a CTA moves itself; past it a second kernel moves them with the
// whole GPU (one launch more, against one CTA's share of the bandwidth).
constexpr int kMaxFusedMoves = 512;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;                // rows of a CTA of the second kernel

// A moved row: where it came from, and its weight and position.
struct __align__(16) Mover {
  int row;
  float weight;
  int pos;
  int to;      // unused by the list; keeps the entry one 16-byte access
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
  int cluster, fused;
};

// Order key of a weight: larger weight, larger key; NaN lowest (but above 0,
// which stands for no row), -0 as 0.  Finite and infinite weights stay below
// kStays.
constexpr uint32_t kStays = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t weight_key(float w) {
  return isnan(w) ? 1u : float_order_key(w + 0.f);
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

// Moves pairs first, first + step, ... < n of (b, g): a warp takes 32 / (d / 4)
// rows at a time, 16 bytes of K or V a lane, four pairs of loads in flight.
__device__ __forceinline__ void move_rows(const EvictParams& p, int bg, int n, int first, int step) {
  const int b = bg / p.G, g = bg - b * p.G;
  const int lane = threadIdx.x & 31;
  const int per = p.d / 4;                     // 16-byte pieces of a row's K and V
  const int at_once = 32 / per, sub = lane / per, piece = lane - sub * per;
  const bool is_v = piece >= per / 2;
  uint16_t* cache = is_v ? p.v : p.k;
  const int off = (is_v ? piece - per / 2 : piece) * 8;
  const Mover* movers = p.movers + static_cast<long long>(bg) * p.half;
  const int32_t* holes = p.holes + static_cast<long long>(bg) * p.half;
  const long long base = static_cast<long long>(bg) * p.C;
  constexpr int U = 4;
  for (int i0 = first * at_once; i0 < n; i0 += step * at_once * U) {
    uint4 x[U];
    long long to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * step * at_once + sub;
      to[u] = -1;
      if (i < n) {
        const int4 raw = __ldcg(reinterpret_cast<const int4*>(movers + i));
        const int hole = __ldcg(holes + i);
        if (piece == 0) {
          p.w_out[base + hole] = __int_as_float(raw.y);
          p.pos_out[base + hole] = raw.z;
        }
        const long long s = row_at(p, b, g, raw.x), t = row_at(p, b, g, hole);
        if (s >= 0 && t >= 0) {
          x[u] = *reinterpret_cast<const uint4*>(cache + s + off);
          to[u] = t;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] >= 0) *reinterpret_cast<uint4*>(cache + to[u] + off) = x[u];
  }
}

// What the CTAs of a cluster tell one another.
struct __align__(16) Shared {
  uint32_t hist[3][kBins];
  int top;                // largest position of the slice
  int fixed;              // rows of the slice that always stay
  int counts[4];          // of the slice: above / at the cut, before / past row n
  int wcounts[kWarps][4]; // of its warps
  int scan[kWarps];
  uint32_t digit;
  int need;
  int red[kWarps];
};

template <bool STASH>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const EvictParams p) {
  __shared__ Shared sh;
  extern __shared__ __align__(16) uint32_t stash[];
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
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  int len = __ldg(p.lens + b);
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
  // this CTA's slice [x0, x1), and each warp's run of it, in whole warps' rows
  const int slice = ((len + cs - 1) / cs + 31) & ~31;
  const int x0 = min(len, rank * slice), x1 = min(len, x0 + slice);
  const bool same_w = wo == w, same_p = po == pos;
  if (n == len) {
    for (int x = x0 + tid; x < x1; x += kThreads) {
      if (!same_w) wo[x] = w[x];
      if (!same_p) po[x] = pos[x];
    }
    return;
  }
  const int run = ((slice + kWarps - 1) / kWarps + 31) & ~31;
  const int y0 = min(x1, x0 + warp * run), y1 = min(x1, y0 + run);
  int* s_pos = reinterpret_cast<int*>(stash);
  uint32_t* s_key = stash + slice;

  // largest position
  int top = INT32_MIN;
#pragma unroll 4
  for (int x = y0 + lane; x < y1; x += 32) {
    const int q = __ldg(pos + x);
    top = max(top, q);
    if (STASH) {
      s_pos[x - x0] = q;
      s_key[x - x0] = __float_as_uint(__ldcg(w + x));
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) sh.red[warp] = top;
  __syncthreads();
  if (tid == 0) {
    for (int i = 0; i < kWarps; ++i) top = max(top, sh.red[i]);
    sh.top = top;
  }
  sync_all();
  for (int r = 0; r < cs; ++r) top = max(top, of_rank(r)->top);

  // Key of row x.  By default rows that always stay come before all; when
  // there are more of them than fit, only they have keys, by weight.
  bool only_fixed = false;
  auto make_key = [&](int q, float wx) -> uint32_t {
    const bool f = stays(p, q, top);
    if (only_fixed) return f ? weight_key(wx) : 0u;
    return f ? kStays : weight_key(wx);
  };
  auto key_at = [&](int x) -> uint32_t {
    if (STASH) return s_key[x - x0];
    return make_key(__ldg(pos + x), __ldcg(w + x));
  };
  auto count_bin = [&](uint32_t* hist, bool in, uint32_t bin) {
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (!m) return;
    const uint32_t lead = __shfl_sync(0xffffffffu, bin, __ffs(m) - 1);
    // equal keys (rows that no query looked at, ties) would queue up on one bin
    if (__all_sync(0xffffffffu, !in || bin == lead)) {
      if (lane == 0) atomicAdd(hist + lead, static_cast<uint32_t>(__popc(m)));
    } else if (in) {
      atomicAdd(hist + bin, 1u);
    }
  };
  // Sums bins [tid * kPer, + kPer) over the cluster and finds the bin that holds
  // the need-th largest key; leaves it in sh.digit and the rank in it in sh.need.
  auto find_digit = [&](int h, int need) {
    uint32_t c[kPer];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) c[i] = 0;
    for (int r = 0; r < cs; ++r) {
      const uint4 v = *reinterpret_cast<const uint4*>(&of_rank(r)->hist[h][tid * kPer]);
      c[0] += v.x;
      c[1] += v.y;
      c[2] += v.z;
      c[3] += v.w;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += c[i];
    // keys in higher bins: an exclusive scan from the top
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_down_sync(0xffffffffu, inc, o);
      if (lane + o < 32) inc += v;
    }
    if (lane == 0) sh.scan[warp] = static_cast<int>(inc);
    __syncthreads();
    uint32_t above = inc - mine;
    for (int i = warp + 1; i < kWarps; ++i) above += static_cast<uint32_t>(sh.scan[i]);
    if (above < static_cast<uint32_t>(need) && above + mine >= static_cast<uint32_t>(need)) {
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) {
        if (above < static_cast<uint32_t>(need) && above + c[i] >= static_cast<uint32_t>(need)) {
          sh.digit = static_cast<uint32_t>(tid * kPer + i);
          sh.need = need - static_cast<int>(above);
        }
        above += c[i];
      }
    }
    __syncthreads();
  };

  // first digit, and the number of rows that always stay
  int fixed = 0;
#pragma unroll 2
  for (int xb = y0; xb < y1; xb += 32) {
    const int x = xb + lane;
    const bool in = x < y1;
    uint32_t key = 0;
    if (in) {
      key = STASH ? make_key(s_pos[x - x0], __uint_as_float(s_key[x - x0])) : key_at(x);
      if (STASH) s_key[x - x0] = key;
    }
    fixed += __popc(__ballot_sync(0xffffffffu, in && key == kStays));
    count_bin(sh.hist[0], in, key >> 21);
  }
  if (lane == 0) sh.red[warp] = fixed;
  __syncthreads();
  if (tid == 0) {
    fixed = 0;
    for (int i = 0; i < kWarps; ++i) fixed += sh.red[i];
    sh.fixed = fixed;
  }
  sync_all();
  fixed = 0;
  for (int r = 0; r < cs; ++r) fixed += of_rank(r)->fixed;
  if (fixed > n) {
    only_fixed = true;
    sync_all();                        // every CTA has read the counts
    for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = 0;
    __syncthreads();
    for (int xb = y0; xb < y1; xb += 32) {
      const int x = xb + lane;
      const bool in = x < y1;
      uint32_t key = 0;
      if (in) {
        key = make_key(__ldg(pos + x), __ldcg(w + x));
        if (STASH) s_key[x - x0] = key;
      }
      count_bin(sh.hist[0], in, key >> 21);
    }
    sync_all();
  }
  find_digit(0, n);
  uint32_t cut = sh.digit << 21;
  int need = sh.need;
#pragma unroll 2
  for (int xb = y0; xb < y1; xb += 32) {
    const int x = xb + lane;
    const uint32_t key = x < y1 ? key_at(x) : 0u;
    count_bin(sh.hist[1], x < y1 && (key >> 21) == (cut >> 21), (key >> 10) & 2047u);
  }
  sync_all();
  find_digit(1, need);
  cut |= sh.digit << 10;
  need = sh.need;
#pragma unroll 2
  for (int xb = y0; xb < y1; xb += 32) {
    const int x = xb + lane;
    const uint32_t key = x < y1 ? key_at(x) : 0u;
    count_bin(sh.hist[2], x < y1 && (key >> 10) == (cut >> 10), key & 1023u);
  }
  sync_all();
  find_digit(2, need);
  cut |= sh.digit;
  need = sh.need;                      // rows equal to the cut that stay, the lowest ones

  // rows above and at the cut, before and past row n
  int c4[4] = {0, 0, 0, 0};
#pragma unroll 2
  for (int xb = y0; xb < y1; xb += 32) {
    const int x = xb + lane;
    const uint32_t key = x < y1 ? key_at(x) : 0u;
    const unsigned gt = __ballot_sync(0xffffffffu, x < y1 && key > cut);
    const unsigned eq = __ballot_sync(0xffffffffu, x < y1 && key == cut);
    const unsigned lo = __ballot_sync(0xffffffffu, x < n);
    c4[0] += __popc(gt & lo);
    c4[1] += __popc(eq & lo);
    c4[2] += __popc(gt & ~lo);
    c4[3] += __popc(eq & ~lo);
  }
  if (lane < 4) sh.wcounts[warp][lane] = lane == 0 ? c4[0] : lane == 1 ? c4[1] : lane == 2 ? c4[2] : c4[3];
  __syncthreads();
  if (tid < 4) {
    int s = 0;
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
  for (int i = 0; i < warp; ++i) {
    const int a = min(x1, x0 + i * run);
    add_run(sh.wcounts[i], rows_before_n(a, min(x1, a + run)), eq_at, hole_at, move_at);
  }
  Mover* movers = p.movers + static_cast<long long>(bg) * p.half;
  int32_t* holes = p.holes + static_cast<long long>(bg) * p.half;
  const unsigned below = (1u << lane) - 1u;
#pragma unroll 2
  for (int xb = y0; xb < y1; xb += 32) {
    const int x = xb + lane;
    const bool in = x < y1;
    const uint32_t key = in ? key_at(x) : 0u;
    const unsigned eq = __ballot_sync(0xffffffffu, in && key == cut);
    const bool keep = in && (key > cut || (key == cut && eq_at + __popc(eq & below) < need));
    eq_at += __popc(eq);
    const bool lo = x < n;
    const unsigned hl = __ballot_sync(0xffffffffu, in && lo && !keep);
    const unsigned mv = __ballot_sync(0xffffffffu, keep && !lo);
    if (in) {
      if (lo) {
        if (keep) {
          if (!same_w) wo[x] = __ldcg(w + x);
          if (!same_p) po[x] = STASH ? s_pos[x - x0] : __ldg(pos + x);
        } else {
          holes[hole_at + __popc(hl & below)] = x;
        }
      } else {
        if (keep)
          movers[move_at + __popc(mv & below)] =
              Mover{x, __ldcg(w + x), STASH ? s_pos[x - x0] : pos[x], 0};
        wo[x] = 0.f;
        po[x] = -1;
      }
    }
    hole_at += __popc(hl);
    move_at += __popc(mv);
  }
  if (!p.fused) {
    if (rank == 0 && tid == 0) p.n_moves[bg] = moves;
    if (cs > 1) cl.sync();             // no CTA leaves while another reads its counts
    return;
  }
  __threadfence();
  sync_all();
  move_rows(p, bg, moves, rank * kWarps + warp, cs * kWarps);
}

// The moves of all (sequence, group)s, kMoveRows a CTA.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int bg = blockIdx.x;
  const int n = __ldcg(p.n_moves + bg);
  const int at_once = 128 / p.d;
  for (long long i0 = static_cast<long long>(blockIdx.y) * kMoveRows; i0 < n;
       i0 += static_cast<long long>(gridDim.y) * kMoveRows) {
    // rows i0 .. i0 + kMoveRows - 1, at_once of them a warp and step
    const int end = static_cast<int>(min(static_cast<long long>(n), i0 + kMoveRows));
    move_rows(p, bg, end, static_cast<int>(i0) / at_once + (threadIdx.x >> 5), kMoveThreads / 32);
  }
}

size_t lists_half(const msa_shape& s) { return static_cast<size_t>(s.seq_kv) / 2; }

struct EvictWs {
  size_t movers, holes, n_moves, bytes;
};

// Holes and movers of a (sequence, group): at most min(n, len - n) <= N / 2 each.
EvictWs ws_layout(const msa_shape& s) {
  const size_t bg = static_cast<size_t>(s.batch) * s.n_kv_heads, lists = bg * lists_half(s);
  EvictWs w{};
  w.movers = 0;
  w.holes = align_up(lists * sizeof(Mover), 256);
  w.n_moves = w.holes + align_up(lists * sizeof(int32_t), 256);
  w.bytes = w.n_moves + align_up(bg * sizeof(int32_t), 256);
  return w;
}

cudaError_t launch_clustered(void (*kernel)(const EvictParams), unsigned grid, int cluster,
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
  // CTAs of a cluster: enough to fill the GPU twice, not below 1024 rows each
  const int64_t bg = static_cast<int64_t>(s.batch) * s.n_kv_heads;
  p.cluster = 1;
  while (p.cluster < kMaxCluster && bg * p.cluster < 2ll * ctx->num_sms &&
         p.C / (2 * p.cluster) >= 1024)
    p.cluster *= 2;
  const int64_t most = std::min<int64_t>(a.budget, std::max(p.C - a.budget, 0));   // moves there can be
  p.fused = most <= static_cast<int64_t>(kMaxFusedMoves) * p.cluster;
  const int64_t slice = align_up(static_cast<size_t>(ceil_div(p.C, p.cluster)), 32);
  const bool stash = slice <= kMaxStash;
  const size_t smem = stash ? static_cast<size_t>(slice) * 8 : 0;
  const unsigned grid = static_cast<unsigned>(bg * p.cluster);
  cudaError_t e = cudaSuccess;
  if (stash)
    e = cudaFuncSetAttribute(evict_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxStash * 8);
  if (e != cudaSuccess) return e;
  {
    ProfScope ps_("cache_evict", st);
    e = launch_clustered(stash ? evict_kernel<true> : evict_kernel<false>, grid, p.cluster, smem, st,
                         p);
  }
  if (e != cudaSuccess || p.fused) return e;
  {
    ProfScope ps_("cache_evict_move", st);
    const int64_t slices = std::min<int64_t>(ceil_div(most, kMoveRows), 65535);   // grid limit
    e = launch_dependent(evict_move_kernel, dim3(static_cast<unsigned>(bg), static_cast<unsigned>(slices)),
                         dim3(kMoveThreads), 0, st, p);
  }
  return e;
}

}  // namespace msa
