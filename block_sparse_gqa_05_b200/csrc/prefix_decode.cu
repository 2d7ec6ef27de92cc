// Decode attention of a batch that shares a prefix, over own caches of
// different lengths, with the softmax weight each own key receives.
//
// The rows of the product are (token, head) pairs of one group.  All rows of
// the batch see the prefix, so its K/V blocks are streamed once per 256 of
// them; the own cache of a (sequence, group) is seen by its T * r rows only.
// A segment is one stream of 128-key blocks:
//   pair    two 128-row tiles of a group over the prefix: both softmax
//           warpgroups work on every block, one tile each;
//   single  one tile (the last one of an odd count, or an own cache): the two
//           warpgroups take alternate blocks, which keeps two blocks in
//           flight and splits the keys between two accumulators.
// The blocks of all segments form one line, weighted by what a block of each
// kind costs, which is cut evenly over a persistent grid of one CTA per SM
// (the lengths are read on the device).  Every (CTA, segment, warpgroup) leaves
// an unnormalised partial output with its running maximum and sum in fp32; a
// second kernel merges them.  With scores wanted, the logits of own keys go to
// the workspace (4 T r bytes per key against 4 d for its K and V) and a third
// kernel turns them into weights once the normalisers are known, which is
// cheaper than reading K again.
//
// In the CTA: warp 0 streams K and V through a ring of tiles by TMA; warps 1
// and 2 load the queries and issue the MMAs of the two warpgroups' tiles (S = Q
// K^T to TMEM, then O += P V with P read from TMEM over S); warp 3 zeroes the V
// rows past a segment's length in its last 16-row step (their weight is zero,
// but 0 * NaN is not; steps past it are neither loaded nor multiplied); warps
// 4..7 and 8..11 are the two softmax warpgroups, one TMEM lane (row) per
// thread.  O is rescaled only when a row's maximum grows by more than 2^8 over
// the one it was accumulated with.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int kThreads = 384;
constexpr int kMaxGrid = 256;      // bound of the persistent grid, for the workspace size
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.f;

// Cost of a block on the line, by the kind of its segment, and of a segment.
constexpr int kCostPair = 5, kCostSingle = 4, kCostSegment = 2;

struct PrefixParams {
  uint16_t* o;
  float* lse;
  const float* w_in;
  float* w_out;
  const int32_t *lens, *prefix_pages, *table;
  uint32_t* err;
  long long* starts;   // [B + 1] line cost of one group of sequences 0 .. b-1
  float* lse2;         // [B*T*H] normalisers, log2
  float2* ml_p;        // [(nsp + grid) * 2, rows_p]  (maximum, sum) of prefix partials
  float* o_p;          // [(nsp + grid) * 2, rows_p, D]
  float2* ml_s;        // [(B*G + grid) * 2, T*r]     of own-cache partials
  float* o_s;          // [(B*G + grid) * 2, T*r, D]
  float* logits;       // [B*G, T*r, 128 nb] (log2 units; scores wanted) or nullptr
  int B, T, H, G, r, C, nb, num_pages;
  int Np, nbp;         // prefix rows and blocks
  int ntile, npt, nsp; // prefix row tiles and tile pairs of a group; prefix segments
  int rows_p, rows_s;  // rows of a prefix / own tile: min(128, B*T*r), T*r
  bool spread_p, spread_s;   // such a tile is there four times, a quarter of the keys each
  bool two_q;          // own queries have two stages, q_stage bytes apart
  int q_stage;
  int grid;
  long long cost_pair, cost_group, cost_prefix;   // of a pair segment, a group's, all prefix segments
  float scale_log2;
};

// Valid rows of sequence b's own cache, clamped into [0, C].
__device__ __forceinline__ int own_len(const PrefixParams& p, int b) {
  const int n = __ldg(p.lens + b);
  if (n >= 0 && n <= p.C) return n;
  atomicOr(p.err, kErrBadLength);
  return n < 0 ? 0 : p.C;
}

__device__ __forceinline__ int blocks_of(int rows) { return (rows + 127) >> 7; }

// Line cost of one group's segment over a sequence's own cache.
__device__ __forceinline__ int own_cost(int nb) { return nb ? nb * kCostSingle + kCostSegment : 0; }

// Line range [cta_begin(c), cta_begin(c + 1)) of CTA c; a block belongs to the
// CTA in whose range it starts.
__device__ __forceinline__ long long cta_begin(long long c, long long total, int grid) {
  return (c * total + grid - 1) / grid;
}
__device__ __forceinline__ int cta_of(long long pos, long long total, int grid) {
  return static_cast<int>(pos * grid / total);
}

// Blocks of a segment that start at ``start`` and cost ``w`` each, up to line
// position ``u``.
__device__ __forceinline__ int blocks_before(long long u, long long start, int w, int nb) {
  if (u <= start) return 0;
  const long long d = u - start;
  return d >= static_cast<long long>(nb) * w ? nb : (static_cast<int>(d) + w - 1) / w;
}

// One CTA's share of a segment.
struct Seg {
  int id;            // index of the segment: prefix segments, then b * G + g
  int j0, n;         // first block and number of blocks
  int nb, rows;      // blocks and valid keys of the whole segment
  int b, g, tile;    // own: sequence and group; prefix: group and first row tile
  bool own, pair;
};

// Walks a CTA's segments along the line, the same way in every role.
struct Walk {
  long long u0, u1, pos;
  int s, b, g, len;

  __device__ __forceinline__ bool next(const PrefixParams& p, Seg& q) {
    for (;;) {
      int w;
      const long long start = pos;
      if (s < p.nsp) {
        q.own = false;
        q.id = s;
        q.g = s / p.npt;
        q.tile = 2 * (s - q.g * p.npt);
        q.pair = q.tile + 1 < p.ntile;
        q.b = 0;
        q.nb = p.nbp;
        q.rows = p.Np;
        w = q.pair ? kCostPair : kCostSingle;
        pos += static_cast<long long>(p.nbp) * w + kCostSegment;
        ++s;
      } else {
        if (b >= p.B) return false;
        if (len < 0) len = own_len(p, b);
        if (len == 0) {
          ++b;
          g = 0;
          len = -1;
          continue;
        }
        q.own = true;
        q.pair = false;
        q.id = p.nsp + b * p.G + g;
        q.b = b;
        q.g = g;
        q.tile = 0;
        q.nb = blocks_of(len);
        q.rows = len;
        w = kCostSingle;
        pos += own_cost(q.nb);
        if (++g == p.G) {
          g = 0;
          ++b;
          len = -1;
        }
      }
      if (start >= u1) return false;
      q.j0 = blocks_before(u0, start, w, q.nb);
      q.n = blocks_before(u1, start, w, q.nb) - q.j0;
      if (q.n > 0) return true;
    }
  }
};

// First of the CTA's blocks of a segment that warpgroup ``wg`` takes, and the
// step to its next one; n0 the number of blocks the CTA had before.  The
// blocks of single segments alternate along the whole walk, so that short
// segments share the warpgroups.
__device__ __forceinline__ int first_block(const Seg& q, int wg, int n0) {
  return q.pair ? 0 : ((n0 ^ wg) & 1);
}
__device__ __forceinline__ int block_step(const Seg& q) { return q.pair ? 1 : 2; }
// Whether the CTA's share ends in a block with rows past the segment's length.
__device__ __forceinline__ bool ragged_end(const Seg& q) {
  return q.j0 + q.n == q.nb && (q.rows & 127) != 0;
}

// 16-row steps of a segment's last block that hold valid rows.
__device__ __forceinline__ int tail_steps(const Seg& q) { return ((q.rows & 127) + 15) >> 4; }

// TMA maps: queries of a prefix tile and of a sequence; K and V in blocks of
// 128 rows and in steps of 16.
struct PrefixMaps {
  CUtensorMap qp, qs, kp, vp, k, v, kp16, vp16, k16, v16;
};

template <int D>
struct PrefixSmem {
  static constexpr uint32_t kTile = 128u * D * 2u;
  static constexpr int kRing = D == 128 ? 5 : 10;       // K or V tiles in the ring
  static constexpr uint32_t kOffRing = 2 * kTile;       // two query tiles first
  static constexpr uint32_t kOffBar = kOffRing + kRing * kTile;
  static constexpr uint32_t kBytes = kOffBar + 512;
};

struct Bars {
  uint64_t *full, *empty;   // [ring] K or V tile loaded / released by both warpgroups
  uint64_t* qfull;          // [2][2] per warpgroup: queries loaded, alternating
  uint64_t* sfull;          // [2] S complete
  uint64_t* pfull;          // [2][2] per warpgroup and half of the keys: P written
  uint64_t *olast, *ofree;  // [2] a segment's O complete / read
  uint64_t* turn;           // [2] of a pair: the warpgroup's turn at the tensor cores
  uint64_t* drain;          // [2] the MMA threads' last commits
};

// Sets *word, after everything this thread (and its warp, before a
// __syncwarp) wrote.
__device__ __forceinline__ void publish_count(const uint32_t* word, uint32_t v) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(word)), "r"(v) : "memory");
}

// Bounded wait until *word >= want (a count another warp publishes).
__device__ __forceinline__ bool wait_count(const uint32_t* word, uint32_t want, volatile int* abort,
                                           uint32_t* err) {
  const uint32_t a = smem_u32(word);
  const uint64_t lim = g_wait_limit_ns;
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    if (static_cast<int32_t>(v - want) >= 0) return true;
    if (it == 0) t0 = globaltimer();
    if (*abort) return false;
    if (lim == 0 || ((it & 63u) == 63u && globaltimer() - t0 > lim)) {
      atomicOr(err, kErrTimeout);
      *abort = 1;
      return false;
    }
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// 32 bytes of one thread to global memory (a whole sector), dst 32-byte aligned.
__device__ __forceinline__ void store8(float* dst, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Keys 64 hf .. 64 hf + 63 of this thread's row of S, those past lim at -inf.
__device__ __forceinline__ void load_half(uint32_t tS, int hf, int lim, bool whole, float* sv) {
  tmem_ld32(tS + hf * 64, sv);
  tmem_ld32(tS + hf * 64 + 32, sv + 32);
  tc_wait_ld();
  if (!whole) {
#pragma unroll
    for (int y = 0; y < 64; ++y) sv[y] = hf * 64 + y <= lim ? sv[y] : -INFINITY;
  }
}

// mbar_wait with a probe before anything else: most waits here are complete.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t phase, volatile int* abort,
                                         uint32_t* err) {
  return mbar_test(bar, phase) || mbar_wait(bar, phase, abort, err);
}

// Waits for K or V tile ``item`` of the ring.  The parity of a slot's phase
// tells its present load from the one before, but not from the one before
// that; a warp that skips tiles (another warpgroup's) may come that early, as
// loads complete in any order.  So it first waits for the load to be issued,
// which happens after the slot's previous tile was loaded and released.
template <int R>
__device__ __forceinline__ bool wait_tile(const Bars& m, const uint32_t* issued, int item,
                                          volatile int* abort, uint32_t* err) {
  return wait_count(issued, static_cast<uint32_t>(item) + 1u, abort, err) &&
         wait_bar(&m.full[item % R], (item / R) & 1, abort, err);
}

// The CTA's range of the line and where its walk starts, by all threads.
// CTA 0 also publishes the sequences' line starts for the merge kernel.
__device__ __forceinline__ void plan(const PrefixParams& p, long long* scratch, Walk* out) {
  const int tid = threadIdx.x;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += own_cost(blocks_of(own_len(p, b)));
  // exclusive scan of the threads' sums
  const int lane = tid & 31, warp = tid >> 5;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  long long before = inc - mine, all = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += scratch[i];
    all += scratch[i];
  }
  const long long total = p.cost_prefix + all * p.G;
  const long long u0 = cta_begin(blockIdx.x, total, p.grid);
  const long long u1 = cta_begin(blockIdx.x + 1, total, p.grid);
  if (blockIdx.x == 0) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      p.starts[b] = at;
      at += own_cost(blocks_of(own_len(p, b)));
    }
    if (tid == 0) p.starts[p.B] = all;
  }
  if (u0 < p.cost_prefix) {
    if (tid == 0) {
      const int g = static_cast<int>(u0 / p.cost_group);
      const long long rest = u0 - g * p.cost_group;
      const int pt = min(static_cast<int>(rest / p.cost_pair), p.npt - 1);
      out->s = g * p.npt + pt;
      out->pos = g * p.cost_group + pt * p.cost_pair;
      out->b = out->g = 0;
      out->len = -1;
    }
  } else {
    if (tid == 0) {            // past every block, unless a thread below finds its place
      out->s = p.nsp;
      out->b = p.B;
      out->g = 0;
      out->len = -1;
      out->pos = total;
    }
    __syncthreads();
    const long long at = u0 - p.cost_prefix;   // < all * G when there is anything left
    if (at >= before * p.G && at < (before + mine) * p.G) {
      long long st = before;
      for (int b = b0; b < b1; ++b) {
        const int c = own_cost(blocks_of(own_len(p, b)));
        if (at < (st + c) * p.G) {
          const int g = static_cast<int>((at - st * p.G) / c);
          out->b = b;
          out->g = g;
          out->pos = p.cost_prefix + st * p.G + static_cast<long long>(g) * c;
          break;
        }
        st += c;
      }
    }
  }
  if (tid == 0) {
    out->u0 = u0;
    out->u1 = u1;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ PrefixMaps tm, const PrefixParams p) {
  using L = PrefixSmem<D>;
  constexpr int R = L::kRing;
  constexpr uint32_t kIdescS = idesc_bf16(128, 128, 0, 0);
  constexpr uint32_t kIdescO = idesc_bf16(128, D, 0, 1);
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long scratch[kThreads / 32];
  __shared__ Walk walk0;
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  Bars m;
  m.full = bars;
  m.empty = bars + R;
  m.qfull = bars + 2 * R;
  m.sfull = m.qfull + 4;
  m.pfull = m.qfull + 6;
  m.olast = m.qfull + 10;
  m.ofree = m.qfull + 12;
  m.turn = m.qfull + 14;
  m.drain = m.qfull + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(m.qfull + 18);
  uint32_t* issued = tmem_slot + 1;                  // K and V tiles whose loads were issued
  uint32_t* fixed = tmem_slot + 2;                   // ragged V tiles zeroed past their length
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 3);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.qfull[2 * i], 1);
      mbar_init(&m.qfull[2 * i + 1], 1);
      mbar_init(&m.sfull[i], 1);
      mbar_init(&m.pfull[2 * i], 128);
      mbar_init(&m.pfull[2 * i + 1], 128);
      mbar_init(&m.olast[i], 1);
      mbar_init(&m.ofree[i], 128);
      mbar_init(&m.turn[i], 1);
      mbar_init(&m.drain[i], 1);
    }
    *issued = *fixed = 0;
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm.qp);
    tma_prefetch_desc(&tm.qs);
    tma_prefetch_desc(&tm.kp);
    tma_prefetch_desc(&tm.vp);
    tma_prefetch_desc(&tm.k);
    tma_prefetch_desc(&tm.v);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  // the kernel may start while the one before it on the stream finishes;
  // nothing of that one's is read or overwritten before this
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  plan(p, scratch, &walk0);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;   // S/P of the warpgroups at 0 and 128, O at 256 and 384
  Walk walk = walk0;
  Seg q;

  if (warp < 4) {
    regs_dec<104>();
    if (warp == 0) {
      // ------------------------------------------------------- K and V tiles
      if (lane == 0) {
        int item = 0;      // tiles issued: K of block n is 2n, V is 2n + 1
        bool ok = true;
        while (ok && walk.next(p, q)) {
          const bool own = q.own || p.prefix_pages;   // which maps
          const bool rag = ragged_end(q);
          for (int j = q.j0; ok && j < q.j0 + q.n; ++j) {
            int y = j * 128, z = q.own ? q.b * p.G + q.g : q.g;
            if (q.own ? p.table != nullptr : p.prefix_pages != nullptr) {
              y = 0;
              z = (q.own ? page_of(p.table, p.nb, p.num_pages, q.b, j, p.err)
                         : page_of(p.prefix_pages, 0, p.num_pages, 0, j, p.err)) *
                      p.G + q.g;
            }
            // of a block with rows past the length only the 16-row steps with valid ones
            const int part = rag && j == q.nb - 1 ? tail_steps(q) : 0;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++item) {
              const int st = item % R;
              if (!(ok = wait_bar(&m.empty[st], ((item / R) & 1) ^ 1, abort_flag, p.err))) break;
              if (!q.pair) mbar_arrive(&m.empty[st]);   // only one warpgroup will release it
              uint8_t* dst = smem + L::kOffRing + st * L::kTile;
              if (part == 0) {
                const CUtensorMap* map = kv ? (own ? &tm.v : &tm.vp) : (own ? &tm.k : &tm.kp);
                mbar_arrive_expect_tx(&m.full[st], L::kTile);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                  tma_load_3d(dst + c * 16384, map, &m.full[st], c * 64, y, z);
              } else {
                const CUtensorMap* map =
                    kv ? (own ? &tm.v16 : &tm.vp16) : (own ? &tm.k16 : &tm.kp16);
                mbar_arrive_expect_tx(&m.full[st], static_cast<uint32_t>(part * 16 * D * 2));
                for (int u = 0; u < part; ++u)
#pragma unroll
                  for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(dst + c * 16384 + u * 2048, map, &m.full[st], c * 64, y + u * 16, z);
              }
              publish_count(issued, static_cast<uint32_t>(item) + 1u);
            }
          }
        }
        // every load issued lands before the CTA may exit
        for (int x = max(0, item - R); x < item; ++x) mbar_drain(&m.full[x % R], (x / R) & 1);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------- V rows past a length, within its last 16 rows
      int n0 = 0;                  // blocks of the segments before
      uint32_t ragged = 0;
      while (walk.next(p, q)) {
        n0 += q.n;
        if (!ragged_end(q)) continue;
        const int item = 2 * n0 - 1;
        const int st = item % R;
        if (!__all_sync(0xffffffffu, wait_tile<R>(m, issued, item, abort_flag, p.err))) break;
        ++ragged;
        const int tail = q.rows & 127, rows = tail_steps(q) * 16 - tail;
        uint8_t* v = smem + L::kOffRing + st * L::kTile + tail * 128;
        for (int x = lane; x < rows * 8; x += 32)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            *reinterpret_cast<uint4*>(v + c * 16384 + x * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) publish_count(fixed, ragged);
      }
    } else {
      // ------------------------- queries and MMAs of one warpgroup's tiles
      const int wg = warp - 1;
      if (lane == 0) {
        const uint32_t tS = tmem + wg * 128, tO = tmem + 256 + wg * 128;
        uint8_t* qbuf = smem + wg * L::kTile;
        const uint32_t ring = smem_u32(smem + L::kOffRing);
        // Queries are loaded one segment ahead.  Own segments use two stages
        // when their rows fit twice; otherwise the tile is free once the
        // softmax has read the segment's last S.
        Walk ahead = walk;
        Seg nq;
        int n0 = 0, n0a = 0, i = 0, jobs = 0, loads = 0, pairs = 0, stage = 0;
        uint32_t ragged = 0;
        auto load_next = [&]() {
          while (ahead.next(p, nq)) {
            const int first = first_block(nq, wg, n0a);
            n0a += nq.n;
            if (first >= nq.n) continue;
            const int sg = nq.own && p.two_q ? loads & 1 : 0;
            uint64_t* bar = &m.qfull[2 * wg + (loads & 1)];
            ++loads;
            const CUtensorMap* map = nq.own ? &tm.qs : &tm.qp;
            const int rows = nq.own ? p.rows_s : p.rows_p;
            const int tok = nq.own ? nq.b * p.T : (nq.tile + (nq.pair ? wg : 0)) * (128 / p.r);
            const int copies = (nq.own ? p.spread_s : p.spread_p) ? 4 : 1;
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(copies * rows * D * 2));
            for (int u = 0; u < copies; ++u)
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(qbuf + sg * p.q_stage + c * 16384 + u * 4096, map, bar, c * 64,
                            nq.g * p.r, tok);
            return;
          }
        };
        load_next();
        bool ok = true;
        while (ok && walk.next(p, q)) {
          const bool rag = ragged_end(q);
          ragged += rag ? 1u : 0u;
          const int first = first_block(q, wg, n0), step = block_step(q);
          if (first < q.n) {
            stage = q.own && p.two_q ? jobs & 1 : 0;
            const uint32_t qa = smem_u32(qbuf + stage * p.q_stage);
            if (!(ok = wait_bar(&m.qfull[2 * wg + (jobs & 1)], (jobs >> 1) & 1, abort_flag, p.err)))
              break;
            const bool early = q.own && p.two_q;
            if (early) load_next();
            // S = Q K^T, over the P that the product before this one has read
            auto issue_s = [&](int x) -> bool {
              const int ki = 2 * (n0 + x), ks_ = ki % R;
              if (!wait_tile<R>(m, issued, ki, abort_flag, p.err)) return false;
              tc_fence_after();
              const uint32_t ka = ring + ks_ * L::kTile;
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
                tc_mma_ss(tS, smem_desc(qa + off, 16, 1024, 2), smem_desc(ka + off, 16, 1024, 2),
                          kIdescS, ks > 0 ? 1u : 0u);
              }
              tc_commit(&m.sfull[wg]);
              tc_commit(&m.empty[ks_]);
              return true;
            };
            if (!(ok = issue_s(first))) break;
            for (int x = first; x < q.n; x += step, ++i) {
              const bool last = x + step >= q.n;
              const int vi = 2 * (n0 + x) + 1, vs_ = vi % R;
              // O += P V, the upper half of the keys first; past a length only
              // the 16-key steps that hold valid rows
              if (x == first && jobs > 0 &&
                  !(ok = wait_bar(&m.ofree[wg], (jobs - 1) & 1, abort_flag, p.err)))
                break;
              if (!(ok = wait_tile<R>(m, issued, vi, abort_flag, p.err))) break;
              int steps = 8;
              if (rag && x == q.n - 1) {
                steps = tail_steps(q);
                if (!(ok = wait_count(fixed, ragged, abort_flag, p.err))) break;
              }
              // Of a pair the two warpgroups take turns at the tensor cores,
              // O += P V and the next S together, so that one is in its
              // softmax while the other's products run
              if (q.pair) {
                if (wg == 0) {
                  if (pairs > 0 &&
                      !(ok = wait_bar(&m.turn[0], (pairs - 1) & 1, abort_flag, p.err)))
                    break;
                } else if (!(ok = wait_bar(&m.turn[1], pairs & 1, abort_flag, p.err))) {
                  break;
                }
                ++pairs;
              }
              const uint32_t va = ring + vs_ * L::kTile;
              uint32_t acc = x > first ? 1u : 0u;
#pragma unroll
              for (int hf = 1; hf >= 0; --hf) {
                if (!(ok = wait_bar(&m.pfull[2 * wg + hf], i & 1, abort_flag, p.err))) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 4 * hf; ks < 4 * hf + 4; ++ks) {
                  if (ks >= steps) break;
                  tc_mma_ts(tO, tS + 64 + ks * 8, smem_desc(va + ks * 16 * 128, 16384, 1024, 2),
                            kIdescO, acc);
                  acc = 1u;
                }
              }
              if (!ok) break;
              tc_commit(&m.empty[vs_]);
              if (last)
                tc_commit(&m.olast[wg]);
              else if (!(ok = issue_s(x + step)))
                break;
              if (q.pair) mbar_arrive(&m.turn[1 - wg]);
            }
            ++jobs;
            if (ok && !early) load_next();
          }
          n0 += q.n;
        }
        // every load and MMA issued completes before TMEM is released
        for (int x = max(0, loads - 2); x < loads; ++x)
          mbar_drain(&m.qfull[2 * wg + (x & 1)], (x >> 1) & 1);
        tc_drain(&m.drain[wg], 0);
      }
      __syncwarp();
    }
  } else {
    regs_inc<192>();
    // ------------------------------------------------------ softmax, one row a thread
    const int wg = (warp >> 2) - 1, quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + wg * 128 + lane_off, tO = tmem + 256 + wg * 128 + lane_off;
    int n0 = 0, i = 0, jobs = 0;
    bool ok = true;
    // The output of a segment is written after the softmax of the next one's
    // first block, so that its last product runs meanwhile.
    bool pend = false, pend_busy = false, pend_valid = false;
    float* pend_o = nullptr;
    auto write_out = [&]() -> bool {
      if (!pend) return true;
      pend = false;
      if (!__all_sync(0xffffffffu, wait_bar(&m.olast[wg], (jobs - 1) & 1, abort_flag, p.err)))
        return false;
      if (pend_busy) {
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          float ov[64];
          tmem_ld32(tO + c * 64, ov);
          tmem_ld32(tO + c * 64 + 32, ov + 32);
          tc_wait_ld();
          if (pend_valid) {
#pragma unroll
            for (int y = 0; y < 64; y += 8) store8(pend_o + c * 64 + y, ov + y);
          }
        }
        tc_fence_before();
      }
      mbar_arrive(&m.ofree[wg]);
      return true;
    };
    while (ok && walk.next(p, q)) {
      const int first = first_block(q, wg, n0), step = block_step(q);
      n0 += q.n;
      // Rows of the tile that exist, this thread's row and its last key.  A tile
      // of few rows is there four times, once per warp, and each warp takes a
      // quarter of every block's keys: four partials.
      const bool spread = q.own ? p.spread_s : p.spread_p;
      const int tile = q.tile + (q.pair ? wg : 0);
      const int nrow = q.own ? p.rows_s : min(128, p.B * p.T * p.r - tile * 128);
      const int row = spread ? lane : quarter * 32 + lane;
      const bool busy = spread || quarter * 32 < nrow;   // a warp without a row only keeps the pace
      const bool valid = row < nrow;
      const int last_key = q.own ? q.rows - p.T + row / p.r : q.rows - 1;
      const long long part =
          2ll * (static_cast<long long>(q.own ? q.id - p.nsp : q.id) + blockIdx.x) + wg;
      const int rows = q.own ? p.rows_s : p.rows_p;
      const long long prow = spread ? (part * 4 + quarter) * rows + row : part * rows + row;
      float2* ml = (q.own ? p.ml_s : p.ml_p) + prow;
      if (first >= q.n) {              // the one block of a short share is the other warpgroup's
        if (valid) *ml = make_float2(-INFINITY, 0.f);
        continue;
      }
      float* logit = nullptr;
      if (q.own && p.logits && valid)
        logit = p.logits + (static_cast<long long>(q.b * p.G + q.g) * p.rows_s + row) * p.nb * 128;
      float mref = -INFINITY, l = 0.f;
      // O of the rows whose maximum outgrew its reference is rescaled; S of a
      // block is issued after the product of the block before, so that one is
      // complete
      auto new_max = [&](float mblk, bool later) {
        const bool grow = valid && mblk > mref + kRescaleLog2;
        if (__any_sync(0xffffffffu, grow && later)) {
          const float a = grow ? fast_exp2(mref - mblk) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float ov[32];
            tmem_ld32(tO + c * 32, ov);
            tc_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) ov[y] *= a;
            tmem_st32(tO + c * 32, ov);
          }
          l *= a;
        }
        if (grow) mref = mblk;
        return mref == -INFINITY ? 0.f : mref;   // a row that has seen no key yet
      };
      for (int x = first; x < q.n; x += step, ++i) {
        if (!(ok = __all_sync(0xffffffffu, wait_bar(&m.sfull[wg], i & 1, abort_flag, p.err)))) break;
        const int j = q.j0 + x;
        const int lim = last_key - j * 128;        // keys past lim are not seen
        const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
        if (spread) {
          tc_fence_after();
          const int k0 = quarter * 32;
          float sv[32];
          tmem_ld32(tS + k0, sv);
          tc_wait_ld();
          if (!__all_sync(0xffffffffu, lim >= k0 + 31)) {
#pragma unroll
            for (int y = 0; y < 32; ++y) sv[y] = k0 + y <= lim ? sv[y] : -INFINITY;
          }
          if (logit) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
              float t8[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) t8[e] = sv[y + e] * p.scale_log2;
              store8(logit + j * 128 + k0 + y, t8);
            }
          }
          float m4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int y = 4; y < 32; y += 2)
            m4[(y >> 1) & 3] = fmax3(m4[(y >> 1) & 3], sv[y], sv[y + 1]);
          const float mu = new_max(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_log2,
                                   x > first);
          const uint64_t mm2 = f2_pack(-mu, -mu);
          uint64_t l2[2] = {0, 0};
          uint32_t pk[16], zero[16];
#pragma unroll
          for (int y = 0; y < 32; y += 2) {
            const float2 e = f2_unpack(ffma2(f2_pack(sv[y], sv[y + 1]), sc2, mm2));
            const float e0 = fast_exp2(e.x), e1 = fast_exp2(e.y);
            pk[y >> 1] = pack2(e0, e1);
            zero[y >> 1] = 0u;
            l2[(y >> 1) & 1] = fadd2(l2[(y >> 1) & 1], f2_pack(e0, e1));
          }
          // this copy's weights of the other warps' keys are zero
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c == quarter)
              tmem_st16(tS + 64 + c * 16, pk);
            else
              tmem_st16(tS + 64 + c * 16, zero);
          }
          const float2 la = f2_unpack(fadd2(l2[0], l2[1]));
          l += la.x + la.y;
          tc_wait_st();
          tc_fence_before();
          mbar_arrive(&m.pfull[2 * wg + 1]);
          mbar_arrive(&m.pfull[2 * wg]);
        } else if (busy) {
          tc_fence_after();
          const bool whole = __all_sync(0xffffffffu, lim >= 127);
          // Half of the row's 128 logits is in registers at a time: keys 0..63
          // for the maximum alone, then 64..127 for both, then 0..63 again
          // (TMEM is read at 4 times the rate at which the rest goes).
          float sv[64];
          float mraw = -INFINITY;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            load_half(tS, hf, lim, whole, sv);
            if (logit) {
#pragma unroll
              for (int y = 0; y < 64; y += 8) {
                float t8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t8[e] = sv[y + e] * p.scale_log2;
                store8(logit + j * 128 + hf * 64 + y, t8);
              }
            }
            float m4[4] = {mraw, sv[0], sv[1], sv[2]};
#pragma unroll
            for (int y = 3; y + 1 < 64; y += 2)
              m4[(y >> 1) & 3] = fmax3(m4[(y >> 1) & 3], sv[y], sv[y + 1]);
            mraw = fmax3(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]), sv[63]);
          }
          const float mu = new_max(mraw * p.scale_log2, x > first);
          const uint64_t mm2 = f2_pack(-mu, -mu);
          uint64_t l2[4] = {0, 0, 0, 0};
          // P goes over the columns of the upper half of S, so that the lower
          // half stays readable
#pragma unroll
          for (int hf = 1; hf >= 0; --hf) {
            if (hf == 0) load_half(tS, 0, lim, whole, sv);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int y = 0; y < 32; y += 2) {
                const float2 e = f2_unpack(ffma2(f2_pack(sv[c * 32 + y], sv[c * 32 + y + 1]), sc2, mm2));
                const float e0 = fast_exp2(e.x), e1 = fast_exp2(e.y);
                pk[y >> 1] = pack2(e0, e1);
                l2[(y >> 1) & 3] = fadd2(l2[(y >> 1) & 3], f2_pack(e0, e1));
              }
              tmem_st16(tS + 64 + hf * 32 + c * 16, pk);
            }
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(&m.pfull[2 * wg + hf]);
          }
          const float2 la = f2_unpack(fadd2(fadd2(l2[0], l2[1]), fadd2(l2[2], l2[3])));
          l += la.x + la.y;
        } else {
          mbar_arrive(&m.pfull[2 * wg + 1]);
          mbar_arrive(&m.pfull[2 * wg]);
        }
        if (x == first && !(ok = write_out())) break;
      }
      if (!ok) break;
      // the partial of this CTA and warpgroup
      if (valid) *ml = make_float2(mref, l);
      pend = true;
      pend_busy = busy;
      pend_valid = valid;
      pend_o = (q.own ? p.o_s : p.o_p) + prow * D;
      ++jobs;
    }
    if (ok) write_out();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Where one row's partials of a segment lie: of CTAs c0 .. c1, at index
// (id + c) * 2 + warpgroup.
struct Parts {
  long long start;
  int c0, n, nb, w, id, row, rows;
  bool own, pair;
  int wg;       // of a pair: the warpgroup of the row's tile
  int sub;      // partials of a warpgroup: 4 of a spread tile, else 1
};

__device__ __forceinline__ Parts parts_of(const PrefixParams& p, long long total, bool own, int b,
                                          int t, int h) {
  Parts s;
  const int g = h / p.r, hr = h - g * p.r;
  s.own = own;
  s.pair = false;
  s.sub = (own ? p.spread_s : p.spread_p) ? 4 : 1;
  s.wg = 0;
  s.w = kCostSingle;
  if (own) {
    s.id = p.nsp + b * p.G + g;
    s.nb = blocks_of(own_len(p, b));
    s.start = p.cost_prefix + p.starts[b] * p.G + static_cast<long long>(g) * own_cost(s.nb);
    s.row = t * p.r + hr;
    s.rows = p.rows_s;
  } else {
    const int at = (b * p.T + t) * p.r + hr, tile = at >> 7, pt = tile >> 1;
    s.id = g * p.npt + pt;
    s.pair = 2 * pt + 1 < p.ntile;
    s.wg = tile & 1;
    s.nb = p.nbp;
    if (s.pair) s.w = kCostPair;
    s.start = g * p.cost_group + pt * p.cost_pair;
    s.row = at & 127;
    s.rows = p.rows_p;
  }
  s.n = 0;
  s.c0 = 0;
  if (s.nb > 0) {
    s.c0 = cta_of(s.start, total, p.grid);
    s.n = 2 * s.sub * (cta_of(s.start + static_cast<long long>(s.nb - 1) * s.w, total, p.grid) - s.c0 + 1);
  }
  return s;
}

// Partial k of the list (two warpgroups a CTA): its index, or -1 when that CTA had no
// block of the segment, or of a pair when it is the other tile's.
__device__ __forceinline__ long long part_at(const PrefixParams& p, const Parts& s, long long total,
                                             int k) {
  const int sub = k & (s.sub - 1), k2 = s.sub == 4 ? k >> 2 : k;
  const int c = s.c0 + (k2 >> 1), wg = k2 & 1;
  const int n = blocks_before(cta_begin(c + 1, total, p.grid), s.start, s.w, s.nb) -
                blocks_before(cta_begin(c, total, p.grid), s.start, s.w, s.nb);
  if (n <= 0 || (s.pair && wg != s.wg)) return -1;
  const long long part = 2ll * ((s.own ? s.id - p.nsp : s.id) + c) + wg;
  return (part * s.sub + sub) * s.rows + s.row;
}

constexpr int kMergeWarps = 8;

// One warp per row (b, t, h): merges its partials.  With m and l the running
// maximum and sum of a partial and O its unnormalised output,
// o = sum 2^(m - M) O / sum 2^(m - M) l, lse = M + log2 of the denominator.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) prefix_merge_kernel(const PrefixParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kMergeWarps + warp;
  if (row >= static_cast<long long>(p.B) * p.T * p.H) return;
  const int h = static_cast<int>(row % p.H);
  const int t = static_cast<int>(row / p.H % p.T), b = static_cast<int>(row / p.H / p.T);
  const long long total = p.cost_prefix + p.starts[p.B] * p.G;
  float M = -INFINITY, den = 0.f;
  bool poison = false;
  constexpr int V = D / 32;
  float acc[V];
#pragma unroll
  for (int y = 0; y < V; ++y) acc[y] = 0.f;
#pragma unroll 1
  for (int own = 0; own < 2; ++own) {
    const Parts s = parts_of(p, total, own != 0, b, t, h);
    const float2* ml = own ? p.ml_s : p.ml_p;
    const float* po = own ? p.o_s : p.o_p;
    for (int k0 = 0; k0 < s.n; k0 += 32) {
      const long long at = k0 + lane < s.n ? part_at(p, s, total, k0 + lane) : -1;
      const float2 v = at >= 0 ? __ldcg(ml + at) : make_float2(-INFINITY, 0.f);
      // fmaxf drops a NaN: a row with a NaN or +inf logit is NaN throughout
      poison |= __any_sync(0xffffffffu, v.x != v.x || v.y != v.y);
      float mx = v.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float Mn = fmaxf(M, mx);
      if (Mn == -INFINITY) continue;
      const float keep = fast_exp2(M - Mn), wgt = at >= 0 ? fast_exp2(v.x - Mn) : 0.f;
      float ls = wgt * v.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      den = den * keep + ls;
#pragma unroll
      for (int y = 0; y < V; ++y) acc[y] *= keep;
      M = Mn;
      unsigned todo = __ballot_sync(0xffffffffu, wgt > 0.f);
      while (todo) {
        // up to four partial rows in flight
        float x[4][V], wk[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int src = todo ? __ffs(todo) - 1 : 0;
          wk[u] = todo ? __shfl_sync(0xffffffffu, wgt, src) : 0.f;
          const long long a = __shfl_sync(0xffffffffu, at, src);
          if (todo) {
            const float* f = po + a * D + lane * V;
            if constexpr (V == 4) {
              const float4 q4 = __ldcg(reinterpret_cast<const float4*>(f));
              x[u][0] = q4.x;
              x[u][1] = q4.y;
              x[u][2] = q4.z;
              x[u][3] = q4.w;
            } else {
              const float2 q2 = __ldcg(reinterpret_cast<const float2*>(f));
              x[u][0] = q2.x;
              x[u][1] = q2.y;
            }
          } else {
#pragma unroll
            for (int y = 0; y < V; ++y) x[u][y] = 0.f;
          }
          todo &= todo - 1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int y = 0; y < V; ++y) acc[y] = fmaf(wk[u], x[u][y], acc[y]);
      }
    }
  }
  if (poison) M = den = __int_as_float(0x7fffffff);
  const float inv = M == -INFINITY ? 0.f : 1.f / den;
  uint16_t* out = p.o + row * D + lane * V;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(out) = pack2(acc[0] * inv, acc[1] * inv);
  if (lane == 0) {
    const float lse2 = M == -INFINITY ? -INFINITY : M + log2f(den);
    p.lse2[row] = lse2;
    if (p.lse) p.lse[row] = lse2 / kLog2e;
  }
}

constexpr int kScoreThreads = 256;

// One thread per own key: the weights its rows gave it, from their logits.
__global__ void __launch_bounds__(kScoreThreads) prefix_score_kernel(const PrefixParams p) {
  __shared__ float norm[128];
  griddep_wait();
  griddep_launch_dependents();
  const int bg = blockIdx.x, b = bg / p.G, g = bg - b * p.G;
  const int len = own_len(p, b);
  if (blockIdx.y * kScoreThreads >= len) return;
  for (int i = threadIdx.x; i < p.rows_s; i += kScoreThreads) {
    const int t = i / p.r;
    const float n = __ldcg(p.lse2 + (static_cast<long long>(b) * p.T + t) * p.H + g * p.r + (i - t * p.r));
    norm[i] = n == -INFINITY ? 0.f : n;     // a row that sees no key has logits of -inf alone
  }
  __syncthreads();
  const long long stride = static_cast<long long>(p.nb) * 128;
  for (int x = blockIdx.y * kScoreThreads + threadIdx.x; x < len; x += gridDim.y * kScoreThreads) {
    const float* s = p.logits + static_cast<long long>(bg) * p.rows_s * stride + x;
    const long long at = static_cast<long long>(bg) * p.C + x;
    float w = 0.f;
#pragma unroll 8
    for (int i = 0; i < p.rows_s; ++i) w += fast_exp2(__ldcg(s + i * stride) - norm[i]);
    p.w_out[at] = (p.w_in ? p.w_in[at] : 0.f) + w;
  }
}

// Most rows of a tile that is spread over the four warps: 32 lie in a warp's
// TMEM lanes; own tiles need them twice, for the next segment's queries.
constexpr size_t kSpreadPrefix = 32, kSpreadOwn = 16;

// Workspace layout.
struct PrefixWs {
  size_t starts, lse2, ml_p, o_p, ml_s, o_s, logits, bytes;
};

PrefixWs ws_layout(const msa_shape& s, bool weights) {
  const size_t r = s.n_q_heads / s.n_kv_heads, d = s.head_dim;
  const size_t rows = static_cast<size_t>(s.batch) * s.seq_q * r;
  const size_t bg = static_cast<size_t>(s.batch) * s.n_kv_heads;
  const size_t nsp = static_cast<size_t>(ceil_div(ceil_div(rows, 128), 2)) * s.n_kv_heads;
  const size_t rp = std::min<size_t>(rows, 128), rs = s.seq_q * r;
  const size_t pr = 2 * (nsp + kMaxGrid) * rp * (rp <= kSpreadPrefix ? 4 : 1);
  const size_t sr = 2 * (bg + kMaxGrid) * rs * (rs <= kSpreadOwn ? 4 : 1);
  PrefixWs w{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t x = at;
    at += align_up(n, 256);
    return x;
  };
  w.starts = take((static_cast<size_t>(s.batch) + 1) * sizeof(long long));
  w.lse2 = take(rows * s.n_kv_heads * sizeof(float));
  w.ml_p = take(pr * sizeof(float2));
  w.o_p = take(pr * d * sizeof(float));
  w.ml_s = take(sr * sizeof(float2));
  w.o_s = take(sr * d * sizeof(float));
  w.logits = take(weights ? bg * s.seq_q * r * ceil_div(s.seq_kv, 128) * 128 * sizeof(float) : 0);
  w.bytes = at;
  return w;
}

template <int D>
cudaError_t launch(const msa_shape& s, const PrefixDecodeArgs& a, const PrefixParams& p,
                   cudaStream_t st) {
  PrefixMaps tm;
  const uint64_t D8 = D;
  const uint64_t dq[3] = {D8, static_cast<uint64_t>(p.H), static_cast<uint64_t>(p.B) * p.T};
  const uint64_t sq[2] = {D8 * 2, static_cast<uint64_t>(p.H) * D * 2};
  const uint32_t bqp[3] = {64, static_cast<uint32_t>(p.r), static_cast<uint32_t>(p.rows_p / p.r)};
  const uint32_t bqs[3] = {64, static_cast<uint32_t>(p.r), static_cast<uint32_t>(p.T)};
  // contiguous: [B*G][C][d]; paged: [num_pages*G][128][d]
  const bool paged = a.pages.table != nullptr;
  const uint64_t rows = paged ? 128 : static_cast<uint64_t>(p.C);
  const uint64_t mats = static_cast<uint64_t>(paged ? p.num_pages : p.B) * p.G;
  const uint64_t dk[3] = {D8, rows, mats};
  const uint64_t sk[2] = {D8 * 2, rows * D * 2};
  const uint32_t bk[3] = {64, 128, 1}, b16[3] = {64, 16, 1};
  const uint64_t dp[3] = {D8, static_cast<uint64_t>(std::max(a.prefix_cap, 1)),
                          static_cast<uint64_t>(p.G)};
  const uint64_t sp[2] = {D8 * 2, dp[1] * D * 2};
  const bool pre = p.Np > 0 && !paged;    // a prefix array of its own
  auto enc = [](CUtensorMap* m, const void* base, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box) {
    return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B);
  };
  bool ok = enc(&tm.qp, a.q, dq, sq, bqp) && enc(&tm.qs, a.q, dq, sq, bqs) &&
            enc(&tm.k, a.k, dk, sk, bk) && enc(&tm.v, a.v, dk, sk, bk) &&
            enc(&tm.k16, a.k, dk, sk, b16) && enc(&tm.v16, a.v, dk, sk, b16);
  if (pre)
    ok = ok && enc(&tm.kp, a.kp, dp, sp, bk) && enc(&tm.vp, a.vp, dp, sp, bk) &&
         enc(&tm.kp16, a.kp, dp, sp, b16) && enc(&tm.vp16, a.vp, dp, sp, b16);
  else
    tm.kp = tm.k, tm.vp = tm.v, tm.kp16 = tm.k16, tm.vp16 = tm.v16;
  if (!ok) return cudaErrorInvalidValue;
  const size_t smem = PrefixSmem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(prefix_attn_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  {
    ProfScope ps_("prefix_attn", st);
    e = launch_dependent(prefix_attn_kernel<D>, dim3(static_cast<unsigned>(p.grid)), dim3(kThreads),
                         smem, st, tm, p);
  }
  if (e != cudaSuccess) return e;
  {
    ProfScope ps_("prefix_merge", st);
    const long long all = static_cast<long long>(p.B) * p.T * p.H;
    e = launch_dependent(prefix_merge_kernel<D>, dim3(static_cast<unsigned>(ceil_div(all, kMergeWarps))),
                         dim3(kMergeWarps * 32), 0, st, p);
  }
  if (e != cudaSuccess || !p.w_out) return e;
  {
    ProfScope ps_("prefix_score", st);
    const int64_t slices = std::min<int64_t>(ceil_div(p.C, kScoreThreads), 65535);   // grid limit
    e = launch_dependent(prefix_score_kernel,
                         dim3(static_cast<unsigned>(p.B) * p.G, static_cast<unsigned>(slices)),
                         dim3(kScoreThreads), 0, st, p);
  }
  return e;
}

}  // namespace

size_t prefix_decode_workspace_bytes(const msa_shape& s, bool weights) {
  return ws_layout(s, weights).bytes;
}

cudaError_t launch_prefix_decode(const msa_shape& s, const PrefixDecodeArgs& a, void* ws,
                                 cudaStream_t st) {
  const DevCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const PrefixWs w = ws_layout(s, a.w_out != nullptr);
  char* base = static_cast<char*>(ws);
  PrefixParams p{};
  p.o = a.o;
  p.lse = a.lse;
  p.w_in = a.w_in;
  p.w_out = a.w_out;
  p.lens = a.lens;
  p.prefix_pages = a.prefix_len > 0 ? a.prefix_pages : nullptr;
  p.table = a.pages.table;
  p.num_pages = a.pages.num_pages;
  p.err = ctx->err;
  p.starts = reinterpret_cast<long long*>(base + w.starts);
  p.lse2 = reinterpret_cast<float*>(base + w.lse2);
  p.ml_p = reinterpret_cast<float2*>(base + w.ml_p);
  p.o_p = reinterpret_cast<float*>(base + w.o_p);
  p.ml_s = reinterpret_cast<float2*>(base + w.ml_s);
  p.o_s = reinterpret_cast<float*>(base + w.o_s);
  p.logits = a.w_out ? reinterpret_cast<float*>(base + w.logits) : nullptr;
  p.B = s.batch;
  p.T = s.seq_q;
  p.H = s.n_q_heads;
  p.G = s.n_kv_heads;
  p.r = s.n_q_heads / s.n_kv_heads;
  p.C = s.seq_kv;
  p.nb = static_cast<int>(ceil_div(s.seq_kv, 128));
  p.Np = a.prefix_len;
  p.nbp = static_cast<int>(ceil_div(a.prefix_len, 128));
  const int64_t rows = static_cast<int64_t>(p.B) * p.T * p.r;
  p.ntile = static_cast<int>(ceil_div(rows, 128));
  p.npt = (p.ntile + 1) / 2;
  p.nsp = p.Np > 0 ? p.npt * p.G : 0;
  p.rows_p = static_cast<int>(std::min<int64_t>(rows, 128));
  p.rows_s = p.T * p.r;
  p.spread_p = rows <= static_cast<int64_t>(kSpreadPrefix);
  p.spread_s = p.rows_s <= static_cast<int>(kSpreadOwn);
  p.two_q = p.rows_s <= 64;
  p.q_stage = p.spread_s ? 16 * 128 : 64 * 128;
  p.cost_pair = static_cast<long long>(p.nbp) * kCostPair + kCostSegment;
  const long long last = (p.ntile & 1) ? static_cast<long long>(p.nbp) * kCostSingle + kCostSegment
                                       : p.cost_pair;
  p.cost_group = (p.npt - 1) * p.cost_pair + last;
  p.cost_prefix = p.Np > 0 ? p.cost_group * p.G : 0;
  p.scale_log2 = kLog2e / sqrtf(static_cast<float>(s.head_dim));
  // no more CTAs than blocks there can be
  const int64_t most = static_cast<int64_t>(p.nsp) * p.nbp + static_cast<int64_t>(p.B) * p.G * p.nb;
  p.grid = static_cast<int>(std::min<int64_t>(most, std::min(std::max(ctx->num_sms, 1), kMaxGrid)));
  return s.head_dim == 128 ? launch<128>(s, a, p, st) : launch<64>(s, a, p, st);
}

cudaError_t set_wait_limit_prefix(uint64_t ns) { return set_wait_limit_here(ns); }

}  // namespace msa
