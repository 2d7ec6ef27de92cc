// Eviction from the own caches by accumulated attention weight.
//
// Per (sequence, group) the n = min(len, budget) best rows stay, under the
// order (rows that always stay, weight descending, row ascending).  With one
// 32-bit order key per row the n-th best key is found by bisection on counts;
// rows above it stay, and of the rows equal to it the lowest ones.  Kept rows
// past n then fill, in order, the dropped rows before n, so only the rows that
// change places are read and written.
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// A moved row: where it came from, and its weight and position.
struct __align__(16) Mover {
  int row;
  float weight;
  int pos;
  int pad;
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
  uint32_t* err;
  int G, C, d, nb, num_pages, budget, n_first, n_recent, half;
};

// Order key of a weight: larger weight, larger key; NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  return isnan(w) ? 0u : float_order_key(w + 0.f);
}

__device__ __forceinline__ bool stays(const EvictParams& p, int pos, int top) {
  return pos < p.n_first || static_cast<long long>(pos) > static_cast<long long>(top) - p.n_recent;
}

// Sum of v over the CTA, to every thread.
__device__ int block_sum(int v, int* scratch) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int i = 0; i < kWarps; ++i) s += scratch[i];
  return s;
}

// Exclusive prefix of f over the CTA's threads; the total in *total.
__device__ int block_rank(bool f, int* scratch, int* total) {
  const unsigned m = __ballot_sync(0xffffffffu, f);
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[warp] = __popc(m);
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kWarps; ++i) {
    before += i < warp ? scratch[i] : 0;
    all += scratch[i];
  }
  *total = all;
  return before + __popc(m & ((1u << (threadIdx.x & 31)) - 1u));
}

// Element offset of row x of (b, g), or -1 (flagged) when its page is bad.
__device__ __forceinline__ long long row_at(const EvictParams& p, int b, int g, int x) {
  if (!p.table) return ((static_cast<long long>(b) * p.G + g) * p.C + x) * p.d;
  const int pg = p.table[static_cast<long long>(b) * p.nb + (x >> 7)];
  if (pg < 0 || pg >= p.num_pages) {
    atomicOr(p.err, kErrBadPage);
    return -1;
  }
  return ((static_cast<long long>(pg) * p.G + g) * 128 + (x & 127)) * p.d;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictParams p) {
  __shared__ int scratch[kWarps];
  const int bg = blockIdx.x, b = bg / p.G, g = bg % p.G;
  const int tid = threadIdx.x;
  int len = p.lens[b];
  if (len < 0 || len > p.C) {
    if (tid == 0) atomicOr(p.err, kErrBadLength);
    len = len < 0 ? 0 : p.C;
  }
  const int n = min(len, p.budget);
  if (g == 0 && tid == 0) p.new_lens[b] = n;
  const long long base = static_cast<long long>(bg) * p.C;
  const float* w = p.w_in + base;
  const int32_t* pos = p.pos_in + base;
  if (n == len) {
    for (int x = tid; x < len; x += kThreads) {
      p.w_out[base + x] = w[x];
      p.pos_out[base + x] = pos[x];
    }
    return;
  }
  int top = INT32_MIN;
  for (int x = tid; x < len; x += kThreads) top = max(top, pos[x]);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) scratch[tid >> 5] = top;
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) top = max(top, scratch[i]);
  int c = 0;
  for (int x = tid; x < len; x += kThreads) c += stays(p, pos[x], top) ? 1 : 0;
  const int fixed = block_sum(c, scratch);
  // Which class the cut falls in, and how many of that class stay: all rows
  // that always stay and need others, or need of those that always stay.
  const bool in_fixed = fixed > n;
  const int need = in_fixed ? n : n - fixed;
  // largest key with at least `need` rows at or above it
  uint32_t cut = 0;
  for (int bit = 31; bit >= 0 && need > 0; --bit) {
    const uint32_t t = cut | (1u << bit);
    c = 0;
    for (int x = tid; x < len; x += kThreads)
      c += (stays(p, pos[x], top) == in_fixed && weight_key(w[x]) >= t) ? 1 : 0;
    if (block_sum(c, scratch) >= need) cut = t;
  }
  c = 0;
  for (int x = tid; x < len; x += kThreads)
    c += (stays(p, pos[x], top) == in_fixed && weight_key(w[x]) > cut) ? 1 : 0;
  const int equal = need - block_sum(c, scratch);   // rows equal to the cut that stay
  int n_eq = 0, n_hole = 0, n_move = 0;
  Mover* movers = p.movers + static_cast<long long>(bg) * p.half;
  int32_t* holes = p.holes + static_cast<long long>(bg) * p.half;
  for (int x0 = 0; x0 < len; x0 += kThreads) {
    const int x = x0 + tid;
    const bool in = x < len;
    const int px = in ? pos[x] : 0;
    const float wx = in ? w[x] : 0.f;
    const bool st = in && stays(p, px, top);
    const uint32_t key = weight_key(wx);
    const bool cls = in && st == in_fixed;
    int total;
    const int re = n_eq + block_rank(cls && key == cut, scratch, &total);
    n_eq += total;
    bool keep = in && (cls ? key > cut || (key == cut && re < equal) : st);
    if (need == 0) keep = in && st;
    const int rh = n_hole + block_rank(in && !keep && x < n, scratch, &total);
    n_hole += total;
    const int rm = n_move + block_rank(keep && x >= n, scratch, &total);
    n_move += total;
    if (!in) continue;
    if (x < n) {
      if (keep) {
        p.w_out[base + x] = wx;
        p.pos_out[base + x] = px;
      } else {
        holes[rh] = x;
      }
    } else {
      if (keep) movers[rm] = Mover{x, wx, px, 0};
      p.w_out[base + x] = 0.f;
      p.pos_out[base + x] = -1;
    }
  }
  __syncthreads();
  const int per = p.d / 8;   // 16-byte pieces of a row
  for (long long i = tid; i < static_cast<long long>(n_move) * per; i += kThreads) {
    const int m = static_cast<int>(i / per), piece = static_cast<int>(i % per);
    const Mover mv = movers[m];
    const int to = holes[m];
    if (piece == 0) {
      p.w_out[base + to] = mv.weight;
      p.pos_out[base + to] = mv.pos;
    }
    const long long s = row_at(p, b, g, mv.row), t = row_at(p, b, g, to);
    if (s < 0 || t < 0) continue;
    reinterpret_cast<uint4*>(p.k + t)[piece] = reinterpret_cast<const uint4*>(p.k + s)[piece];
    reinterpret_cast<uint4*>(p.v + t)[piece] = reinterpret_cast<const uint4*>(p.v + s)[piece];
  }
}

size_t lists_half(const msa_shape& s) { return static_cast<size_t>(s.seq_kv) / 2; }

}  // namespace

// Holes and movers of a (sequence, group): at most min(n, len - n) <= N / 2 each.
size_t evict_workspace_bytes(const msa_shape& s) {
  const size_t lists = static_cast<size_t>(s.batch) * s.n_kv_heads * lists_half(s);
  return align_up(lists * sizeof(Mover), 256) + align_up(lists * sizeof(int32_t), 256) + 256;
}

cudaError_t launch_cache_evict(const msa_shape& s, const EvictArgs& a, void* ws, cudaStream_t st) {
  const DevCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const size_t lists = static_cast<size_t>(s.batch) * s.n_kv_heads * lists_half(s);
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
  p.movers = static_cast<Mover*>(ws);
  p.holes = reinterpret_cast<int32_t*>(static_cast<char*>(ws) +
                                       align_up(lists * sizeof(Mover), 256));
  p.err = ctx->err;
  p.G = s.n_kv_heads;
  p.C = s.seq_kv;
  p.d = s.head_dim;
  p.nb = static_cast<int>(ceil_div(s.seq_kv, 128));
  p.budget = a.budget;
  p.n_first = a.n_first;
  p.n_recent = a.n_recent;
  p.half = static_cast<int>(lists_half(s));
  {
    ProfScope ps_("cache_evict", st);
    evict_kernel<<<static_cast<unsigned>(s.batch) * s.n_kv_heads, kThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace msa
