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
// (the lengths are read on the device: a warp of each CTA walks its part of the
// line and hands the others one descriptor a segment, as five copies of the
// walk made the code too large for the instruction cache).  Every (CTA, segment, warpgroup) leaves
// an unnormalised partial output with its running maximum and sum in fp32; a
// second kernel merges them.  With scores wanted, the logits of own keys go to
// the workspace and other CTAs of that kernel turn them into weights: 4 T r bytes
// a key written and read, against 2 d to read K again and its product.  Measured
// at T r = 8 and d = 128 (64 bytes against 256: 16 of 110 us for 16 caches of
// 16,384); from T r = d / 4 on the logits are the more bytes.
//
// In the CTA: warp 0 streams K and V through a ring of tiles by TMA; warps 1
// and 2 load the queries and issue the MMAs of the two warpgroups' tiles (S = Q
// K^T to TMEM, then O += P V with P read from TMEM over S), and zero the V rows
// past a segment's length in its last 16-row step (their weight is zero, but
// 0 * NaN is not; steps past it are neither loaded nor multiplied); warp 3 walks
// the line; warps 4..7 and 8..11 are the two softmax warpgroups, one TMEM lane
// (row) per thread.  O is rescaled only when a row's maximum grows by more than
// 2^8 over the one it was accumulated with.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int kThreads = 384;
// Most rows of a tile that is spread over the four warps: 32 lie in a warp's
// TMEM lanes; own tiles need them twice, for the next segment's queries.  And
// the blocks a segment needs to be spread: its softmax is then twice as fast,
// but it leaves four partials instead of one.
constexpr size_t kSpreadPrefix = 32, kSpreadOwn = 16;
constexpr int kSpreadBlocks = 4;
constexpr int kMaxGrid = 256;      // bound of the persistent grid, for the workspace size
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.f;   // a row's reference follows its maximum when that is 2^8 above it

// Cost of a block on the line, in some 220 clocks: of a pair, of a spread tile, of
// another single tile of up to 32 rows and of more; and of a segment.  Measured on
// 32 sequences with a prefix of 8192 (the CTAs of a finer line end together: 52 to
// 50 us) and on 24 with 5 tokens each, whose own tiles have 40 rows (18 for these
// against 16: 112 and 115 us).
constexpr int kCostPair = 16, kCostSpread = 10, kCostFew = 16, kCostSingle = 18, kCostSegment = 4,
              kCostPairSegment = 28;
constexpr int kCostMost = 18;

struct PrefixParams {
  uint16_t* o;
  float* lse;
  const float* w_in;
  float* w_out;
  const int32_t *lens, *prefix_pages, *table;
  const uint16_t* v;   // own caches
  uint32_t* err;
  int2* dropped;       // [B*G] whether the last block and the one before left out values of V (T > 1)
  int2* span;          // [nsp + B*G] first and last CTA with blocks of a segment
  float2* ml_p;        // [(nsp + grid) * 2, rows_p]  (maximum, sum) of prefix partials
  float* o_p;          // [(nsp + grid) * 2, rows_p, D]
  float2* ml_s;        // [(B*G + grid) * 2, T*r]     of own-cache partials
  float* o_s;          // [(B*G + grid) * 2, T*r, D]
  float* logits;       // [B*G, T*r, 128 nb] (log2 units; scores wanted) or nullptr
  int B, T, H, G, r, C, nb, num_pages;
  int grid;            // CTAs of the attention
  int Np, nbp;         // prefix rows and blocks
  int ntile, npt, nsp; // prefix row tiles and tile pairs of a group; prefix segments
  int rows_p, rows_s;  // rows of a prefix / own tile: min(128, B*T*r), T*r
  bool spread_p, spread_s;   // rows few enough for the tile to be there four times, a quarter of the keys each
  bool two_q;          // own queries have two stages, q_stage bytes apart
  int q_stage;
  int cost_pair, cost_group, cost_prefix;   // line cost of a pair segment, a group's, all prefix segments
  float scale_log2;
};

// Valid rows of sequence b's own cache, clamped into [0, C].  Read from L2, as the
// scores are: the kernel before on the stream may still run when this one starts
// and write them (an eviction's new lengths) after this SM cached the line.
__device__ __forceinline__ int own_len(const PrefixParams& p, int b) {
  const int n = __ldcg(p.lens + b);
  if (n >= 0 && n <= p.C) return n;
  atomicOr(p.err, kErrBadLength);
  return n < 0 ? 0 : p.C;
}

__device__ __forceinline__ int blocks_of(int rows) { return (rows + 127) >> 7; }

// The line is cut into ``parts`` ranges [part_begin(c), part_begin(c + 1)); a
// block belongs to the range it starts in.
__device__ __forceinline__ int part_begin(int c, int total, int parts) {
  const int q = total / parts;
  return c * q + min(c, total - q * parts);
}

// Blocks of a segment that start at ``start`` and cost ``w`` each, up to line
// position ``u``.
__device__ __forceinline__ int blocks_before(int u, int start, int w, int nb) {
  return u <= start ? 0 : min(nb, (u - start + w - 1) / w);
}

// Whether a segment of nb blocks is spread over the four warps.
__device__ __forceinline__ bool spreads(const PrefixParams& p, bool own, int nb) {
  return (own ? p.spread_s : p.spread_p) && nb >= kSpreadBlocks;
}

// Whether the tiles of a kind have 32 rows or fewer.
__device__ __forceinline__ bool few_rows(const PrefixParams& p, bool own) {
  return (own ? p.rows_s : p.rows_p) <= 32;
}

// Line cost of a block of a single segment, and of one group's own segment.
__device__ __forceinline__ int single_cost(const PrefixParams& p, bool own, int nb) {
  return spreads(p, own, nb) ? kCostSpread : few_rows(p, own) ? kCostFew : kCostSingle;
}
__device__ __forceinline__ int own_cost(const PrefixParams& p, int nb) {
  return nb ? nb * single_cost(p, true, nb) + kCostSegment : 0;
}

// One CTA's share of a segment, as the walk hands it on (n == 0: the end).
struct __align__(16) Seg {
  int id;          // index of the segment: prefix segments, then b * G + g
  int j0, n;       // first block and number of blocks
  int rows;        // valid keys of the whole segment
  int b, g;        // own: sequence and group; prefix: group
  int tile_kind;   // prefix: first row tile << 2; | kPair | kOwn
  int n0;          // blocks of the CTA before
  __device__ __forceinline__ bool own() const { return (tile_kind & 1) != 0; }
  __device__ __forceinline__ bool pair() const { return (tile_kind & 2) != 0; }
  __device__ __forceinline__ int tile() const { return tile_kind >> 2; }
  // First of these blocks that warpgroup wg takes, and the step to its next
  // one.  The blocks of single segments alternate along the whole walk, so that
  // short segments share the warpgroups.
  __device__ __forceinline__ int first(int wg) const { return pair() ? 0 : ((n0 ^ wg) & 1); }
  __device__ __forceinline__ int step() const { return pair() ? 1 : 2; }
  // Whether the share ends in a block with rows past the segment's length, and
  // the 16-row steps of that block that hold valid rows.
  __device__ __forceinline__ bool ragged() const {
    return j0 + n == ((rows + 127) >> 7) && (rows & 127) != 0;
  }
  __device__ __forceinline__ int tail_steps() const { return ((rows & 127) + 15) >> 4; }
};

// Walks a CTA's segments along the line, by a whole warp: runs of sequences without
// rows (idle slots of a batch) are passed 32 at a time, as one by one a few million
// of them took longer than the other warps wait.
struct Walk {
  int u0, u1, pos;
  int s, b, g, len, n0;

  __device__ __forceinline__ Seg next(const PrefixParams& p) {
    Seg q;
    for (;;) {
      int w, nb;
      const int start = pos;
      if (start >= u1) break;
      if (s < p.nsp) {
        const int g_ = s / p.npt, tile = 2 * (s - g_ * p.npt);
        const bool pair = tile + 1 < p.ntile;
        q.id = s;
        q.b = 0;
        q.g = g_;
        q.tile_kind = tile << 2 | (pair ? 2 : 0);
        q.rows = p.Np;
        nb = p.nbp;
        w = pair ? kCostPair : single_cost(p, false, nb);
        pos += nb * w + (pair ? kCostPairSegment : kCostSegment);
        ++s;
      } else {
        if (len < 0) {
          const int at = b + static_cast<int>(threadIdx.x & 31);
          const int n = at < p.B ? own_len(p, at) : 0;
          const unsigned some = __ballot_sync(0xffffffffu, n > 0);
          if (!some) {
            b += 32;
            if (b >= p.B) break;      // not before u1
            continue;
          }
          const int first = __ffs(some) - 1;
          len = __shfl_sync(0xffffffffu, n, first);
          b += first;
        }
        q.id = p.nsp + b * p.G + g;
        q.b = b;
        q.g = g;
        q.tile_kind = 1;
        q.rows = len;
        nb = blocks_of(len);
        w = single_cost(p, true, nb);
        pos += own_cost(p, nb);
        if (++g >= p.G) {
          g = 0;
          ++b;
          len = -1;
        }
      }
      q.j0 = blocks_before(u0, start, w, nb);
      q.n = blocks_before(u1, start, w, nb) - q.j0;
      q.n0 = n0;
      if (q.n > 0) {
        n0 += q.n;
        if (q.j0 == 0) p.span[q.id].x = blockIdx.x;
        if (q.j0 + q.n == nb) p.span[q.id].y = blockIdx.x;
        return q;
      }
    }
    q.n = 0;
    return q;
  }
};

// TMA maps: queries of a prefix tile and of a sequence; K and V in blocks of
// 128 rows and in steps of 16.
struct PrefixMaps {
  CUtensorMap qp, qs, kp, vp, k, v, kp16, vp16, k16, v16;
};

constexpr int kSegRing = 8;        // descriptors the walk is ahead at most

template <int D>
struct PrefixSmem {
  static constexpr uint32_t kTile = 128u * D * 2u;
  static constexpr int kRing = D == 128 ? 5 : 10;       // K or V tiles in the ring
  static constexpr uint32_t kOffRing = 2 * kTile;       // two query tiles first
  static constexpr uint32_t kOffBar = kOffRing + kRing * kTile;
  static constexpr uint32_t kOffSeg = kOffBar + (2 * kRing + 2 * kSegRing + 16) * 8 + 16;
  static constexpr uint32_t kOffPlan = kOffSeg + kSegRing * 32;      // scan scratch, first segment
  static constexpr uint32_t kBytes = kOffPlan + kThreads / 32 * 4 + 64;
};

struct Bars {
  uint64_t *full, *empty;   // [ring] K or V tile loaded / released by both warpgroups
  uint64_t *dfull, *dempty; // [kSegRing] descriptor written / read by all
  uint64_t* qfull;          // [2][2] per warpgroup: queries loaded, alternating
  uint64_t* sfull;          // [2] S complete
  uint64_t* pfull;          // [2] P written
  uint64_t *olast, *ofree;  // [2] a segment's O complete / read
  uint64_t* turn;           // [2] of a pair: the warpgroup's turn at the tensor cores
  uint64_t* drain;          // [2] the MMA warps' last commits
};

// What the waits need; limit: in clocks; 0 makes a wait that is not complete at
// its first probe expire.
struct Waits {
  volatile int* abort;
  uint32_t* err;
  long long limit;
};

// The waits' limit in clocks, at 2 GHz, just above what the SM runs at.
__device__ __forceinline__ long long wait_clocks() {
  const uint64_t ns = g_wait_limit_ns;
  return static_cast<long long>(ns > (1ull << 61) ? 1ull << 62 : 2 * ns);
}

__device__ __forceinline__ bool give_up(const Waits& w) {
  atomicOr(w.err, kErrTimeout);
  *w.abort = 1;
  return false;
}

// Bounded wait for the completion of phase ``phase`` (parity), as mbar_wait, with
// the SM clock for the bound: reading the timer takes longer than most waits.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t phase, const Waits& w) {
  if (w.limit == 0 ? mbar_test(bar, phase) : mbar_try_wait(bar, phase)) return true;
  const long long t0 = clock64();
  do {
    if (w.limit != 0 && mbar_try_wait(bar, phase)) return true;
    if (*w.abort) return false;
  } while (clock64() - t0 < w.limit);
  return give_up(w);
}
// The same for a whole warp.  All lanes probe: measured, a hand-over between two
// warps takes 100 clocks so, 190 through one lane and a shuffle.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase, const Waits& w) {
  return __all_sync(0xffffffffu, wait_bar(bar, phase, w)) != 0;
}

// Sets *word, after everything this thread (and its warp, before a
// __syncwarp) wrote.
__device__ __forceinline__ void publish_count(const uint32_t* word, uint32_t v) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(word)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t read_count(const uint32_t* word) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(word)) : "memory");
  return v;
}
// Bounded wait until *word >= want (a count another warp publishes).
__device__ __forceinline__ bool wait_count(const uint32_t* word, uint32_t want, const Waits& w) {
  if (static_cast<int32_t>(read_count(word) - want) >= 0) return true;
  const long long t0 = clock64();
  do {
    if (w.limit != 0 && static_cast<int32_t>(read_count(word) - want) >= 0) return true;
    if (*w.abort) return false;
  } while (clock64() - t0 < w.limit);
  return give_up(w);
}

// Waits for K or V tile ``item`` of the ring.  The parity of a slot's phase
// tells its present load from the one before, but not from the one before
// that; a warp that skips tiles (another warpgroup's) may come that early, as
// loads complete in any order.  So it first waits for the load to be issued,
// which happens after the slot's previous tile was loaded and released.
template <int R>
__device__ __forceinline__ bool warp_wait_tile(const Bars& m, const uint32_t* issued, int item,
                                               const Waits& w) {
  const bool ok = wait_count(issued, static_cast<uint32_t>(item) + 1u, w) &&
                  wait_bar(&m.full[item % R], (item / R) & 1, w);
  return __all_sync(0xffffffffu, ok) != 0;
}

__device__ __forceinline__ Seg read_seg(const Seg* at) {
  Seg q;
  reinterpret_cast<int4*>(&q)[0] = reinterpret_cast<const int4*>(at)[0];
  reinterpret_cast<int4*>(&q)[1] = reinterpret_cast<const int4*>(at)[1];
  return q;
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

// Logits of keys past lim to -inf.
template <int N>
__device__ __forceinline__ void mask_keys(float* sv, int lim) {
  if (__all_sync(0xffffffffu, lim >= N - 1)) return;
#pragma unroll
  for (int y = 0; y < N; ++y) sv[y] = y <= lim ? sv[y] : -INFINITY;
}

template <int N>
__device__ __forceinline__ float max_keys(const float* sv) {
  float m4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
  for (int y = 4; y < N; y += 2) m4[(y >> 1) & 3] = fmax3(m4[(y >> 1) & 3], sv[y], sv[y + 1]);
  return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
}

// N logits in units of log2 to the workspace.
template <int N>
__device__ __forceinline__ void store_logits(float* dst, const float* sv, float scale_log2) {
#pragma unroll
  for (int y = 0; y < N; y += 8) {
    float t8[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t8[e] = sv[y + e] * scale_log2;
    store8(dst + y, t8);
  }
}

// 32 weights 2^(s scale - m) as bf16 pairs, and their sums in fp32.
__device__ __forceinline__ void exp_keys(const float* sv, uint64_t sc2, uint64_t mm2, uint32_t* pk,
                                         uint64_t* l2) {
#pragma unroll
  for (int y = 0; y < 32; y += 2) {
    const float2 e = f2_unpack(ffma2(f2_pack(sv[y], sv[y + 1]), sc2, mm2));
    const float e0 = fast_exp2(e.x), e1 = fast_exp2(e.y);
    pk[y >> 1] = pack2(e0, e1);
    l2[(y >> 1) & 3] = fadd2(l2[(y >> 1) & 3], f2_pack(e0, e1));
  }
}

// Whether either bf16 of a word is an infinity or a NaN; and the word with zeros for them.
__device__ __forceinline__ bool not_finite2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// Rows [y0, y1) of the V tile of an own block, which not all of the T queries of the
// sequence see.  Their weight is 0 there, but 0 times an infinity or a NaN is not: a
// warp sets these to zero and returns whether there were any, for the finishing
// kernel to add them where they are seen.
template <int D>
__device__ __forceinline__ bool drop_not_finite(uint8_t* tile, int y0, int y1) {
  bool any = false;
#pragma unroll 1
  for (int u = y0 * 8 + static_cast<int>(threadIdx.x & 31); u < y1 * 8; u += 32)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint4* at = reinterpret_cast<uint4*>(tile + c * 16384) + u;
      const uint4 w = *at;
      if (not_finite2(w.x) || not_finite2(w.y) || not_finite2(w.z) || not_finite2(w.w)) {
        *at = make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
        any = true;
      }
    }
  return __any_sync(0xffffffffu, any) != 0;
}

// A value all lanes of the warp hold, in the form the compiler knows as such.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// MMAs and commits by one elected lane (always the same one) of a whole warp,
// without a branch: descriptors then stay in uniform registers, which the
// instructions read; under a branch on the lane each of them was moved there
// first (8 MMAs of S: 690 clocks against 512 of execution).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar))
      : "memory");
}

// The CTA's range of the line and where its walk starts, by all threads.
__device__ __forceinline__ void plan(const PrefixParams& p, int* scratch, Walk* out) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += own_cost(p, blocks_of(own_len(p, b)));
  // exclusive scan of the threads' sums: in the warps, then over their totals
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  int sums = lane < kWarps ? scratch[lane] : 0;
  const int own_total = sums;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += v;
  }
  const int before = inc - mine + __shfl_sync(0xffffffffu, sums - own_total, warp);
  const int all = __shfl_sync(0xffffffffu, sums, kWarps - 1);
  const int total = p.cost_prefix + all * p.G;
  // no more parts than blocks there are: every part between a segment's first
  // and last one then holds a block of it
  const int parts = max(1, min(static_cast<int>(gridDim.x), total / kCostMost));
  const int u0 = min(total, part_begin(blockIdx.x, total, parts));
  const int u1 = min(total, part_begin(blockIdx.x + 1, total, parts));
  if (tid == 0) {
    out->u0 = u0;
    out->u1 = u1;
    out->n0 = out->b = out->g = 0;
    out->len = -1;
    if (u0 < p.cost_prefix) {
      const int g = u0 / p.cost_group, pt = min((u0 - g * p.cost_group) / p.cost_pair, p.npt - 1);
      out->s = g * p.npt + pt;
      out->pos = g * p.cost_group + pt * p.cost_pair;
    } else {                   // past every block, unless a thread below finds its place
      out->s = p.nsp;
      out->b = p.B;
      out->pos = total;
    }
  }
  __syncthreads();
  const int at = u0 - p.cost_prefix;   // < all * G when there is anything left
  if (at >= 0 && at >= before * p.G && at < (before + mine) * p.G) {
    int st = before;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int c = own_cost(p, blocks_of(own_len(p, b)));
      if (at < (st + c) * p.G) {
        const int g = (at - st * p.G) / c;
        out->b = b;
        out->g = g;
        out->pos = p.cost_prefix + st * p.G + g * c;
        break;
      }
      st += c;
    }
  }
}

// MANY: T > 1, with V rows that some queries of the sequence do not see.  Compiled
// apart: the look at them costs the one token nothing (32 sequences with a prefix of
// 8192 48.4 against 47.7 us in one kernel) and 24 of 5 tokens 1.4 in 114.
template <int D, bool MANY>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ PrefixMaps tm, const __grid_constant__ PrefixParams p) {
  using L = PrefixSmem<D>;
  constexpr int R = L::kRing;
  constexpr uint32_t kIdescS = idesc_bf16(128, 128, 0, 0);
  constexpr uint32_t kIdescO = idesc_bf16(128, D, 0, 1);
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  Bars m;
  m.full = bars;
  m.empty = bars + R;
  m.dfull = bars + 2 * R;
  m.dempty = m.dfull + kSegRing;
  m.qfull = m.dempty + kSegRing;
  m.sfull = m.qfull + 4;
  m.pfull = m.qfull + 6;
  m.olast = m.qfull + 8;
  m.ofree = m.qfull + 10;
  m.turn = m.qfull + 12;
  m.drain = m.qfull + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(m.qfull + 16);
  uint32_t* issued = tmem_slot + 1;                  // K and V tiles whose loads were issued
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);
  Seg* segs = reinterpret_cast<Seg*>(smem + L::kOffSeg);
  int* scratch = reinterpret_cast<int*>(smem + L::kOffPlan);
  Walk* walk0 = reinterpret_cast<Walk*>(scratch + kThreads / 32);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 2);
    }
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(&m.dfull[i], 1);
      mbar_init(&m.dempty[i], 11);       // the TMA, MMA and softmax warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.qfull[2 * i], 1);
      mbar_init(&m.qfull[2 * i + 1], 1);
      mbar_init(&m.sfull[i], 1);
      mbar_init(&m.pfull[i], 4);         // a tile's softmax warps
      mbar_init(&m.olast[i], 1);
      mbar_init(&m.ofree[i], 4);
      mbar_init(&m.turn[i], 1);
      mbar_init(&m.drain[i], 1);
    }
    *issued = 0;
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
  plan(p, scratch, walk0);
  __syncthreads();
  tc_fence_after();
  const Waits w{abort_flag, p.err, wait_clocks()};
  const uint32_t tmem = *tmem_slot;   // S/P of the warpgroups at 0 and 128, O at 256 and 384

  if (warp < 4) {
    regs_dec<88>();        // 4 x 88 + 8 x 208 warps' worth is what the launch has; with 80 these spilled
    if (warp == 3) {
      // ------------------------------------------------------------ the walk
      Walk walk = *walk0;
      for (int k = 0;; ++k) {
        const Seg q = walk.next(p);
        const int slot = k % kSegRing;
        if (!warp_wait(&m.dempty[slot], ((k / kSegRing) & 1) ^ 1, w)) break;
        if (lane == 0) {
          reinterpret_cast<int4*>(segs + slot)[0] = reinterpret_cast<const int4*>(&q)[0];
          reinterpret_cast<int4*>(segs + slot)[1] = reinterpret_cast<const int4*>(&q)[1];
          mbar_arrive(&m.dfull[slot]);
        }
        __syncwarp();
        if (q.n == 0) break;
      }
    } else if (warp == 0) {
      // ------------------------------------------------------- K and V tiles
      if (lane == 0) {
        int item = 0;      // tiles issued: K of block n is 2n, V is 2n + 1
        bool ok = true;
        for (int k = 0; ok; ++k) {
          const int ds = k % kSegRing;
          if (!wait_bar(&m.dfull[ds], (k / kSegRing) & 1, w)) break;
          const Seg q = read_seg(segs + ds);
          if (q.n == 0) break;
          mbar_arrive(&m.dempty[ds]);
          const bool own = q.own();
          const int32_t* table = own ? p.table + static_cast<long long>(q.b) * p.nb : p.prefix_pages;
          const bool paged = own ? p.table != nullptr : p.prefix_pages != nullptr;
          const bool kv_own = own || paged;           // which maps
          const bool rag = q.ragged();
          for (int j = q.j0; ok && j < q.j0 + q.n; ++j) {
            int y = j * 128, z = own ? q.b * p.G + q.g : q.g;
            if (paged) {
              y = 0;
              z = page_of(table, 0, p.num_pages, 0, j, p.err) * p.G + q.g;
            }
            // of a block with rows past the length only the 16-row steps with valid ones
            const int part = rag && j == q.j0 + q.n - 1 ? q.tail_steps() : 0;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv, ++item) {
              const int st = item % R;
              if (!(ok = wait_bar(&m.empty[st], ((item / R) & 1) ^ 1, w))) break;
              if (!q.pair()) mbar_arrive(&m.empty[st]);   // only one warpgroup will release it
              uint8_t* dst = smem + L::kOffRing + st * L::kTile;
              const CUtensorMap* map = kv_own ? (kv ? &tm.v : &tm.k) : (kv ? &tm.vp : &tm.kp);
              if (part == 0) {
                mbar_arrive_expect_tx(&m.full[st], L::kTile);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                  tma_load_3d(dst + c * 16384, map, &m.full[st], c * 64, y, z);
              } else {
                map += &tm.k16 - &tm.k;               // the same in 16-row steps
                mbar_arrive_expect_tx(&m.full[st], static_cast<uint32_t>(part * 16 * D * 2));
#pragma unroll 1
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
    } else {
      // ------------------------- queries and MMAs of one warpgroup's tiles
      const int wg = static_cast<int>(uniform(warp - 1));
      const uint32_t tS = uniform(tmem) + wg * 128, tO = tS + 256;
      uint8_t* qbuf = smem + wg * L::kTile;
      const uint32_t ring = smem_u32(smem + L::kOffRing);
      int ka = 0, i = 0, jobs = 0, loads = 0, pairs = 0;
      // Loads the queries of the warpgroup's next segment, if its descriptor is
      // there (descriptors ka.. were not looked at).  Own segments use two
      // stages when their rows fit twice and are loaded one ahead; otherwise
      // the tile is free once the softmax has read the segment's last S.
      auto load_next = [&](int k) {
        for (; ka < k + kSegRing; ++ka) {
          const int ds = ka % kSegRing;
          bool there = false;
          if (lane == 0) there = mbar_test(&m.dfull[ds], (ka / kSegRing) & 1);
          __syncwarp();
          if (!__shfl_sync(0xffffffffu, there, 0)) return;
          const Seg a = read_seg(segs + ds);
          if (a.n == 0) return;
          if (a.first(wg) >= a.n) continue;
          if (lane == 0) {
            const bool own = a.own();
            uint64_t* bar = &m.qfull[2 * wg + (loads & 1)];
            uint8_t* dst = qbuf + (own && p.two_q ? (loads & 1) * p.q_stage : 0);
            const CUtensorMap* map = own ? &tm.qs : &tm.qp;
            const int rows = own ? p.rows_s : p.rows_p;
            const int tok = own ? a.b * p.T : (a.tile() + (a.pair() ? wg : 0)) * (128 / p.r);
            const int copies = spreads(p, own, blocks_of(a.rows)) ? 4 : 1;
            if (copies == 1 && few_rows(p, own)) dst += wg * 64 * 128;   // rows 64.. of the tile
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(copies * rows * D * 2));
#pragma unroll 1
            for (int u = 0; u < copies; ++u)
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(dst + c * 16384 + u * 4096, map, bar, c * 64, a.g * p.r, tok);
          }
          __syncwarp();
          ++loads;
          ++ka;
          return;
        }
      };
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int ds = k % kSegRing;
        if (!(ok = warp_wait(&m.dfull[ds], (k / kSegRing) & 1, w)))
          break;
        const Seg q = read_seg(segs + ds);
        if (q.n == 0) break;
        const int first = q.first(wg), step = q.step();
        if (first < q.n) {
          const bool early = q.own() && p.two_q;
          if (loads == jobs) {
            ka = k;
            load_next(k);
          }
          ka = max(ka, k + 1);
          if (!(ok = warp_wait(&m.qfull[2 * wg + (jobs & 1)], (jobs >> 1) & 1, w)))
            break;
          if (early) load_next(k);
          const uint64_t qd =
              smem_desc(uniform(smem_u32(qbuf) + (early ? (jobs & 1) * p.q_stage : 0)), 16, 1024, 2);
          const bool rag = q.ragged(), pair = q.pair();
          // first block with V rows to clean: past the length, or not seen by every query
          const int clean = MANY && q.own() ? (max(q.rows - p.T + 1, 0) >> 7) - q.j0 : rag ? q.n - 1 : q.n;
          // S = Q K^T of block x, over the P that the product before has read
          auto wait_k = [&](int x) {
            return warp_wait_tile<R>(m, issued, 2 * (q.n0 + x), w);
          };
          auto issue_s = [&](int x) {
            const int st = 2 * (q.n0 + x) % R;
            const uint64_t kd = smem_desc(uniform(ring + st * L::kTile), 16, 1024, 2);
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
              mma_ss(tS, qd + off, kd + off, kIdescS, ks > 0 ? 1u : 0u);
            }
            mma_commit(&m.sfull[wg]);
            mma_commit(&m.empty[st]);
          };
          if (!(ok = wait_k(first))) break;
          issue_s(first);
          for (int x = first; x < q.n; x += step, ++i) {
            const bool last = x + step >= q.n;
            // O += P V; past a length only the 16-key steps that hold valid rows
            if (x == first && jobs > 0 &&
                !(ok = warp_wait(&m.ofree[wg], (jobs - 1) & 1, w)))
              break;
            const int item = 2 * (q.n0 + x) + 1, st = item % R;
            if (!(ok = warp_wait_tile<R>(m, issued, item, w)))
              break;
            uint8_t* v = smem + L::kOffRing + st * L::kTile;
            int steps = 8;
            if (x >= clean) {
              if (rag && x == q.n - 1) {
                steps = q.tail_steps();
                const int tail = q.rows & 127, units = (steps * 16 - tail) * 8;
                for (int y = lane; y < units; y += 32)
#pragma unroll
                  for (int c = 0; c < D / 64; ++c)
                    *reinterpret_cast<uint4*>(v + c * 16384 + tail * 128 + y * 16) =
                        make_uint4(0, 0, 0, 0);
              }
              const bool some = MANY && q.own();
              const int j = q.j0 + x;
              bool any = false;
              if (some) any = drop_not_finite<D>(v, max(q.rows - p.T + 1 - j * 128, 0), min(q.rows - j * 128, 128));
              fence_proxy_async_smem();
              __syncwarp();
              // after the fence, which would wait for it
              if (some && lane == 0) (&p.dropped[q.id - p.nsp].x)[blocks_of(q.rows) - 1 - j] = any;
            }
            // Of a pair the two warpgroups take turns at the tensor cores, O +=
            // P V and the next S together, so that one is in its softmax while
            // the other's products run; the weights are waited for last
            if (pair) {
              if (!last && !(ok = wait_k(x + step))) break;
              if ((wg == 1 || pairs > 0) &&
                  !(ok = warp_wait(&m.turn[wg], (pairs - 1 + wg) & 1, w)))
                break;
              ++pairs;
            }
            const uint64_t vd = smem_desc(uniform(smem_u32(v)), 16384, 1024, 2);
            if (!(ok = warp_wait(&m.pfull[wg], i & 1, w))) break;
            tc_fence_after();
            if (steps == 8) {
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                mma_ts(tO, tS + ks * 8, vd + ks * 128, kIdescO, x > first || ks > 0 ? 1u : 0u);
            } else {
#pragma unroll 1
              for (int ks = 0; ks < steps; ++ks)
                mma_ts(tO, tS + ks * 8, vd + ks * 128, kIdescO, x > first || ks > 0 ? 1u : 0u);
            }
            mma_commit(&m.empty[st]);
            if (last) {
              mma_commit(&m.olast[wg]);
            } else {
              if (!pair && !(ok = wait_k(x + step))) break;
              issue_s(x + step);
            }
            if (pair && lane == 0) mbar_arrive(&m.turn[1 - wg]);
            __syncwarp();
          }
          ++jobs;
          if (ok && loads == jobs) load_next(k);
        }
        if (lane == 0) mbar_arrive(&m.dempty[ds]);
      }
      // every load and MMA issued completes before TMEM is released
      mma_commit(&m.drain[wg]);
      for (int x = max(0, loads - 2); x < loads; ++x)
        mbar_drain(&m.qfull[2 * wg + (x & 1)], (x >> 1) & 1);
      mbar_drain(&m.drain[wg], 0);
    }
  } else {
    regs_inc<208>();
    // ------------------------------------------------------ softmax, one row a thread
    const int wg = (warp >> 2) - 1, quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + wg * 128 + lane_off, tO = tmem + 256 + wg * 128 + lane_off;
    const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
    int i = 0, jobs = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int ds = k % kSegRing;
      if (!(ok = warp_wait(&m.dfull[ds], (k / kSegRing) & 1, w)))
        break;
      const Seg q = read_seg(segs + ds);
      __syncwarp();
      if (q.n == 0) break;
      if (lane == 0) mbar_arrive(&m.dempty[ds]);
      const int first = q.first(wg), step = q.step();
      const bool own = q.own();
      // Rows of the tile that exist, this thread's row and its last key.  A tile
      // of few rows is there four times, once per warp, and each warp takes a
      // quarter of every block's keys: four partials.
      const bool spread = spreads(p, own, blocks_of(q.rows));
      const int tile = q.tile() + (q.pair() ? wg : 0);
      const int nrow = own ? p.rows_s : min(128, p.B * p.T * p.r - tile * 128);
      // (a tile of up to 32 rows has them in the third quarter for the second
      // warpgroup: the working warps of the two then run on different schedulers)
      const int q0 = few_rows(p, own) ? 2 * wg : 0;
      const int row = spread ? lane : (quarter - q0) * 32 + lane;
      const bool valid = row >= 0 && row < nrow;
      const bool busy = spread || (quarter >= q0 && (quarter - q0) * 32 < nrow);   // others keep the pace
      const int last_key = own ? q.rows - p.T + row / p.r : q.rows - 1;
      const long long part = 2ll * (static_cast<long long>(own ? q.id - p.nsp : q.id) + blockIdx.x) + wg;
      const int rows = own ? p.rows_s : p.rows_p;
      const bool room = own ? p.spread_s : p.spread_p;     // partials lie four times as far apart
      const long long prow = (room ? part * 4 + (spread ? quarter : 0) : part) * rows + row;
      float2* ml = (own ? p.ml_s : p.ml_p) + prow;
      if (first >= q.n) {              // the one block of a short share is the other warpgroup's
        if (valid) *ml = make_float2(-INFINITY, 0.f);
        continue;
      }
      float* logit = nullptr;
      if (own && p.logits && valid)
        logit = p.logits + (static_cast<long long>(q.b * p.G + q.g) * p.rows_s + row) * p.nb * 128;
      float mref = -INFINITY, l = 0.f;   // reference of the accumulated O, sum of the weights
      for (int x = first; x < q.n; x += step, ++i) {
        if (!(ok = warp_wait(&m.sfull[wg], i & 1, w))) break;
        const int j = q.j0 + x;
        const int lim = last_key - j * 128;        // keys past lim are not seen
        if (busy) {
          tc_fence_after();
          // O of the rows whose maximum is above their reference by more than
          // 2^8 is rescaled to a new one; S of a block is issued after the
          // product of the block before, so that one is complete
          auto new_reference = [&](float top) {
            const bool grow = valid && top > mref + kRescaleLog2;
            if (!__any_sync(0xffffffffu, grow)) return;
            const float a = grow ? fast_exp2(mref - top) : 1.f;
            if (x > first) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                float ov[32];
                tmem_ld32(tO + c * 32, ov);
                tc_wait_ld();
#pragma unroll
                for (int y = 0; y < 32; ++y) ov[y] *= a;
                tmem_st32(tO + c * 32, ov);
              }
            }
            l *= a;
            if (grow) mref = top;
          };
          uint64_t l2[4] = {0, 0, 0, 0};
          uint32_t pk[16];
          if (spread) {
            const int k0 = quarter * 32;
            float sv[32];
            tmem_ld32(tS + k0, sv);
            tc_wait_ld();
            mask_keys<32>(sv, lim - k0);
            if (logit) store_logits<32>(logit + j * 128 + k0, sv, p.scale_log2);
            new_reference(max_keys<32>(sv) * p.scale_log2);
            const float mu = mref == -INFINITY ? 0.f : mref;   // a row that has seen no key yet
            exp_keys(sv, sc2, f2_pack(-mu, -mu), pk, l2);
            // this copy's weights of the other warps' keys are zero
            uint32_t zero[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) zero[y] = 0u;
#pragma unroll 1
            for (int c = 1; c < 4; ++c) tmem_st16(tS + ((quarter + c) & 3) * 16, zero);
            tmem_st16(tS + quarter * 16, pk);
          } else {
            // The whole row in registers: one wait for TMEM, and nothing between
            // the exponentials, whose unit is what bounds a block (1,024 clocks)
            float sv[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sv + c * 32);
            tc_wait_ld();
            mask_keys<128>(sv, lim);
            if (logit) store_logits<128>(logit + j * 128, sv, p.scale_log2);
            new_reference(max_keys<128>(sv) * p.scale_log2);
            const float mu = mref == -INFINITY ? 0.f : mref;
            const uint64_t mm2 = f2_pack(-mu, -mu);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              exp_keys(sv + c * 32, sc2, mm2, pk, l2);
              tmem_st16(tS + c * 16, pk);
            }
          }
          const float2 la = f2_unpack(fadd2(fadd2(l2[0], l2[1]), fadd2(l2[2], l2[3])));
          l += la.x + la.y;
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.pfull[wg]);
      }
      if (!ok) break;
      // the partial of this CTA and warpgroup; the S of the next segment's first
      // block is on its way meanwhile
      if (!(ok = warp_wait(&m.olast[wg], jobs++ & 1, w))) break;
      if (busy) {
        tc_fence_after();
        float ov[D];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32(tO + c * 32, ov + c * 32);
        tc_wait_ld();
        tc_fence_before();
        if (valid) {
          float* orow = (own ? p.o_s : p.o_p) + prow * D;
#pragma unroll
          for (int y = 0; y < D; y += 8) store8(orow + y, ov + y);
          *ml = make_float2(mref, l);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.ofree[wg]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kMergeWarps = 8;

// The partials of one row of a segment: n of them, of the CTAs of its span, of
// both warpgroups (of a pair: the tile's), of the four quarters of a spread tile.
struct Parts {
  int n, per, first;     // per CTA; index of the first CTA's first (CTA, warpgroup)
  int rows, at;          // rows of a partial, and this row's place
  bool spread, room;     // room: partials lie four times as far apart
};

__device__ __forceinline__ Parts parts_of(const PrefixParams& p, bool own, int tok, int b, int h, int len) {
  Parts s;
  const int g = h / p.r, hr = h - g * p.r;
  s.room = own ? p.spread_s : p.spread_p;
  s.rows = own ? p.rows_s : p.rows_p;
  const int nb = own ? blocks_of(len) : p.nbp;
  s.spread = spreads(p, own, nb);
  int id, wgs = 2, wg0 = 0;
  if (own) {
    id = b * p.G + g;
    s.at = (tok - b * p.T) * p.r + hr;
  } else {
    const int at = tok * p.r + hr, tile = at >> 7;
    id = g * p.npt + (tile >> 1);
    s.at = at & 127;
    if ((tile | 1) < p.ntile) {
      wgs = 1;
      wg0 = tile & 1;
    }
  }
  s.per = wgs * (s.spread ? 4 : 1);
  s.n = 0;
  s.first = 0;
  if (nb > 0) {
    // A CTA whose wait expired leaves without the spans of its other segments:
    // what the workspace held there is no index.  One within the grid is, as the
    // partials of every segment have room for that of every CTA.
    const int2 span = __ldcg(p.span + (own ? p.nsp + id : id));
    if (span.x >= 0 && span.x <= span.y && span.y < p.grid) {
      s.n = (span.y - span.x + 1) * s.per;
      s.first = 2 * (id + span.x) + wg0;
    } else {
      atomicOr(p.err, kErrTimeout);
    }
  }
  return s;
}

// Index of the row in partial k.
__device__ __forceinline__ int part_row(const Parts& s, int k) {
  const int c = k / s.per, in = k - c * s.per;
  const int part = s.first + 2 * c + (s.spread ? in >> 2 : in);
  return (s.room ? part * 4 + (s.spread ? in & 3 : 0) : part) * s.rows + s.at;
}

// Partials k0 + lane of a row: adds them to the row's maximum and sum, and
// returns the lane's weight 2^(m - M); *keep is what scales what was added
// before, *at the lane's partial row, or -1 when that saw no key (and may never have
// been written).  A NaN of a partial (a logit was NaN or +inf) makes *den NaN: the
// maximum drops it, the sums do not.
__device__ __forceinline__ float add_norm(const float2* ml, const Parts& s, int k, int* at, float* M,
                                          float* den, float* keep) {
  float2 v = make_float2(-INFINITY, 0.f);
  *at = -1;
  if (k < s.n) {
    const int row = part_row(s, k);
    v = __ldcg(ml + row);
    if (v.x != -INFINITY) *at = row;
  }
  float mx = v.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float Mn = fmaxf(*M, mx), base = Mn == -INFINITY ? 0.f : Mn;
  *keep = fast_exp2(*M - base);
  const float w = fast_exp2(v.x - base);
  float l = w * v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  *den = *den * *keep + l;
  *M = Mn;
  return w;
}

// Adds to a lane's columns of the output of query t what drop_not_finite left out
// of the rows that it sees: a weight times an infinity or a NaN is that itself.
template <int V>
__device__ __forceinline__ void add_not_finite(const PrefixParams& p, int b, int g, int t, int len, float* acc) {
  const int lane = static_cast<int>(threadIdx.x & 31);
#pragma unroll 1
  for (int x = max(len - p.T + 1, 0); x <= len - p.T + t; ++x) {
    const long long row =
        p.table ? (static_cast<long long>(page_of(p.table, p.nb, p.num_pages, b, x >> 7, p.err)) * p.G + g) * 128 +
                      (x & 127)
                : (static_cast<long long>(b) * p.G + g) * p.C + x;
    const uint32_t* v = reinterpret_cast<const uint32_t*>(p.v + row * (V * 32) + lane * V);
#pragma unroll
    for (int c = 0; c < V / 2; ++c) {
      const uint32_t w = __ldcg(v + c);
      if ((w & 0x7f80u) == 0x7f80u) acc[2 * c] += __uint_as_float(w << 16);
      if ((w & 0x7f800000u) == 0x7f800000u) acc[2 * c + 1] += __uint_as_float(w & 0xffff0000u);
    }
  }
}

// The last CTAs merge the partials: o = sum 2^(m - M) O / sum 2^(m - M) l and
// lse = M + log2 of the denominator, kMergeWarps / split rows a CTA, split
// warps sharing a row's partials (few rows have many).  The first add the
// weights of ``keys`` own keys of a (sequence, group), from their logits and
// the normalisers of the rows, which each finds for itself: a few hundred
// cached loads, against one launch more and its wait.  MANY: as above.
template <int D, bool MANY>
__global__ void __launch_bounds__(kMergeWarps * 32)
    prefix_finish_kernel(const __grid_constant__ PrefixParams p, int merge_ctas, int split, int keys) {
  constexpr int V = D / 32;
  __shared__ __align__(16) float buf[kMergeWarps * 128];   // merge: D a warp; scores: 4 a thread
  __shared__ float norm[128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int score_ctas = static_cast<int>(gridDim.x) - merge_ctas;
  if (static_cast<int>(blockIdx.x) >= score_ctas) {
    const int sub = warp % split;
    const long long row = (static_cast<long long>(blockIdx.x - score_ctas) * kMergeWarps + warp) / split;
    const bool in = row < static_cast<long long>(p.B) * p.T * p.H;
    const int tok = in ? static_cast<int>(row / p.H) : 0, h = in ? static_cast<int>(row % p.H) : 0;
    const int b = tok / p.T, len = own_len(p, b);
    griddep_wait();
    griddep_launch_dependents();
    int dropped = 0;
    if (MANY && len > 0) {
      const int2 d = __ldcg(p.dropped + b * p.G + h / p.r);
      dropped = d.x | (len - p.T + 1 < ((len - 1) & ~127) ? d.y : 0);   // unset when one block has all such rows
    }
    float acc[V];
#pragma unroll
    for (int y = 0; y < V; ++y) acc[y] = 0.f;
    float M = -INFINITY, den = 0.f;
#pragma unroll 1
    for (int own = 0; own < 2; ++own) {
      const Parts s = parts_of(p, own != 0, tok, b, h, len);
      const float* po = (own ? p.o_s : p.o_p) + lane * V;
#pragma unroll 1
      for (int k0 = 0; k0 < s.n; k0 += 32) {
        int at;
        float keep;
        const float w = add_norm(own ? p.ml_s : p.ml_p, s, k0 + lane, &at, &M, &den, &keep);
#pragma unroll
        for (int y = 0; y < V; ++y) acc[y] *= keep;
        // (one whose weight is rounded to 0 too: 0 times its infinities is not 0)
        unsigned todo = __ballot_sync(0xffffffffu, at >= 0 && (lane & (split - 1)) == sub);
        while (todo) {
          constexpr int U = 8;         // partial rows in flight
          float x[U][V], wk[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int src = todo ? __ffs(todo) - 1 : 0;
            wk[u] = __shfl_sync(0xffffffffu, w, src);
            const int a = __shfl_sync(0xffffffffu, at, src);
            if (todo) {
              const float* f = po + static_cast<long long>(a) * D;
              if constexpr (V == 4)
                *reinterpret_cast<float4*>(x[u]) = __ldcg(reinterpret_cast<const float4*>(f));
              else
                *reinterpret_cast<float2*>(x[u]) = __ldcg(reinterpret_cast<const float2*>(f));
            } else {
              wk[u] = 0.f;
#pragma unroll
              for (int y = 0; y < V; ++y) x[u][y] = 0.f;
            }
            todo &= todo - 1;
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int y = 0; y < V; ++y) acc[y] = fmaf(wk[u], x[u][y], acc[y]);
        }
      }
    }
    if (split > 1) {
#pragma unroll
      for (int y = 0; y < V; ++y) buf[warp * D + lane * V + y] = acc[y];
      __syncthreads();
      if (sub != 0) return;
#pragma unroll 1
      for (int u = 1; u < split; ++u)
#pragma unroll
        for (int y = 0; y < V; ++y) acc[y] += buf[(warp + u) * D + lane * V + y];
    }
    if (!in) return;
    if (MANY && dropped) add_not_finite<V>(p, b, h / p.r, tok - b * p.T, len, acc);
    const bool none = M == -INFINITY && den == 0.f;
    const float inv = none ? 0.f : 1.f / den;
    uint16_t* out = p.o + row * D + lane * V;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(out) =
          make_uint2(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(out) = pack2(acc[0] * inv, acc[1] * inv);
    if (lane == 0 && p.lse) p.lse[row] = none ? -INFINITY : (M + log2f(den)) / kLog2e;
    return;
  }
  // a thread: four keys, and one of 4 * 256 / keys shares of the rows
  const int id = static_cast<int>(blockIdx.x);
  const int chunks = (p.C + keys - 1) / keys;
  const int bg = id / chunks, b = bg / p.G, g = bg - b * p.G;
  const int len = own_len(p, b), x0 = (id - bg * chunks) * keys;
  griddep_wait();
  griddep_launch_dependents();
  if (x0 >= len) return;
  // normalisers: a lane per row, the warps share its partials
#pragma unroll 1
  for (int i0 = 0; i0 < p.rows_s; i0 += 32) {
    const int i = i0 + lane, t = i / p.r;
    float M = -INFINITY, den = 0.f;
    if (i < p.rows_s) {
#pragma unroll 1
      for (int own = 0; own < 2; ++own) {
        const Parts s = parts_of(p, own != 0, b * p.T + t, b, g * p.r + i - t * p.r, len);
        const float2* ml = own ? p.ml_s : p.ml_p;
#pragma unroll 4
        for (int k = warp; k < s.n; k += kMergeWarps) {
          const float2 v = __ldcg(ml + part_row(s, k));
          const float Mn = fmaxf(M, v.x), base = Mn == -INFINITY ? 0.f : Mn;
          den = den * fast_exp2(M - base) + fast_exp2(v.x - base) * v.y;
          M = Mn;
        }
      }
    }
    __syncthreads();
    buf[warp * 64 + lane] = M;
    buf[warp * 64 + 32 + lane] = den;
    __syncthreads();
    if (warp == 0 && i < p.rows_s) {
      M = -INFINITY;
      den = 0.f;
#pragma unroll
      for (int u = 0; u < kMergeWarps; ++u) M = fmaxf(M, buf[u * 64 + lane]);
      const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int u = 0; u < kMergeWarps; ++u) den += buf[u * 64 + 32 + lane] * fast_exp2(buf[u * 64 + lane] - base);
      // a row that sees no key has logits of -inf alone
      norm[i] = M == -INFINITY && den == 0.f ? 0.f : M + log2f(den);
    }
  }
  __syncthreads();
  // 1024 keys at a time (fewer when threads share the rows: then once)
  const int quads = min(keys, 1024) / 4, share = static_cast<int>(threadIdx.x) / quads;
  const int shares = kMergeWarps * 32 / quads, quad = static_cast<int>(threadIdx.x) - share * quads;
  const size_t stride = static_cast<size_t>(p.nb) * 128;
#pragma unroll 1
  for (int x1 = x0; x1 < min(len, x0 + keys); x1 += 4 * quads) {
    const int x = x1 + 4 * quad;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (x < len) {
      const float* s = p.logits + static_cast<size_t>(bg) * p.rows_s * stride + x;
#pragma unroll 8
      for (int i = share; i < p.rows_s; i += shares) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(s + i * stride));
        const float n = norm[i];
        w.x += fast_exp2(v.x - n);
        w.y += fast_exp2(v.y - n);
        w.z += fast_exp2(v.z - n);
        w.w += fast_exp2(v.w - n);
      }
    }
    if (shares > 1) {
      float4* sums = reinterpret_cast<float4*>(buf);
      if (share > 0) sums[threadIdx.x - quads] = w;
      __syncthreads();
      if (share > 0) return;
      for (int u = 0; u + 1 < shares; ++u) {
        const float4 v = sums[u * quads + quad];
        w.x += v.x;
        w.y += v.y;
        w.z += v.z;
        w.w += v.w;
      }
    }
    const long long at = static_cast<long long>(bg) * p.C + x;
    const float we[4] = {w.x, w.y, w.z, w.w};
    const float* old = p.w_in + at;
    float* to = p.w_out + at;
    if (x + 3 < len && ((reinterpret_cast<uintptr_t>(old) | reinterpret_cast<uintptr_t>(to)) & 15u) == 0) {
      if (p.w_in) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(old));
        w = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
      }
      *reinterpret_cast<float4*>(to) = w;
      continue;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)      // rows of C elements need not be 16-byte aligned
      if (x + e < len) to[e] = (p.w_in ? __ldcg(old + e) : 0.f) + we[e];
  }
}

// Workspace layout, from its start rounded up to kWsAlign: the caller's is a
// multiple of 16 bytes, and store8 needs 32.
constexpr size_t kWsAlign = 32;
struct PrefixWs {
  size_t span, dropped, ml_p, o_p, ml_s, o_s, logits, bytes;
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
  w.span = take((nsp + bg) * sizeof(int2));
  w.dropped = take(s.seq_q > 1 ? bg * sizeof(int2) : 0);
  w.ml_p = take(pr * sizeof(float2));
  w.o_p = take(pr * d * sizeof(float));
  w.ml_s = take(sr * sizeof(float2));
  w.o_s = take(sr * d * sizeof(float));
  w.logits = take(weights ? bg * s.seq_q * r * ceil_div(s.seq_kv, 128) * 128 * sizeof(float) : 0);
  w.bytes = at + kWsAlign - 16;
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
  const auto attn = p.T > 1 ? prefix_attn_kernel<D, true> : prefix_attn_kernel<D, false>;
  const auto finish = p.T > 1 ? prefix_finish_kernel<D, true> : prefix_finish_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(attn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  {
    ProfScope ps_("prefix_attn", st);
    e = launch_dependent(attn, dim3(static_cast<unsigned>(p.grid)), dim3(kThreads), smem, st, tm, p);
  }
  if (e != cudaSuccess) return e;
  // warps a row: enough to have some 8 warps on every SM (with 16, two sequences
  // of 8 heads took 11.2 against 10.7 us, 32 of 64 52.7 against 52.0)
  const int64_t all = static_cast<int64_t>(p.B) * p.T * p.H;
  int split = 1;
  while (split < kMergeWarps && all * split < 8ll * p.grid) split *= 2;
  const int64_t merge = ceil_div(all * split, kMergeWarps);
  // keys of a scoring CTA: of short caches with many rows fewer, 4 threads sharing
  // the rows (700 keys of 40 rows 112 against 126 us; 1024 keys of 8 rows 49.4
  // against 48.3, so these have whole CTAs); of long ones two rounds (16,384 keys
  // of 8 rows 111.5 against 113.6 us, with four 121.8)
  const int keys = p.C <= 1024 && p.rows_s > 16 ? 256 : p.C >= 8192 ? 2048 : 1024;
  const int64_t score = p.w_out ? static_cast<int64_t>(p.B) * p.G * ceil_div(p.C, keys) : 0;
  if (merge + score >= (1ll << 31)) return cudaErrorInvalidValue;
  ProfScope ps_("prefix_finish", st);
  return launch_dependent(finish, dim3(static_cast<unsigned>(merge + score)), dim3(kMergeWarps * 32), 0, st, p,
                          static_cast<int>(merge), split, keys);
}

}  // namespace

// The line's positions and the partials' row indices are 32-bit.
bool prefix_decode_supported(const msa_shape& s, int prefix_len) {
  const int64_t r = s.n_q_heads / s.n_kv_heads, rows = static_cast<int64_t>(s.batch) * s.seq_q * r;
  const int64_t bg = static_cast<int64_t>(s.batch) * s.n_kv_heads;
  const int64_t nsp = ceil_div(ceil_div(rows, 128), 2) * s.n_kv_heads;
  const int64_t line = nsp * (ceil_div(prefix_len, 128) * kCostMost + kCostPairSegment) +
                       bg * (ceil_div(s.seq_kv, 128) * kCostMost + kCostSegment);
  const int64_t parts = std::max(2 * (nsp + kMaxGrid) * 128, 2 * (bg + kMaxGrid) * std::max<int64_t>(s.seq_q * r, 64));
  return line < (1ll << 31) && parts < (1ll << 31);
}

size_t prefix_decode_workspace_bytes(const msa_shape& s, bool weights) {
  return ws_layout(s, weights).bytes;
}

cudaError_t launch_prefix_decode(const msa_shape& s, const PrefixDecodeArgs& a, void* ws,
                                 cudaStream_t st) {
  const DevCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const PrefixWs w = ws_layout(s, a.w_out != nullptr);
  char* base = reinterpret_cast<char*>(align_up(reinterpret_cast<uintptr_t>(ws), kWsAlign));
  PrefixParams p{};
  p.o = a.o;
  p.lse = a.lse;
  p.w_in = a.w_in;
  p.w_out = a.w_out;
  p.lens = a.lens;
  p.v = a.v;
  p.prefix_pages = a.prefix_len > 0 ? a.prefix_pages : nullptr;
  p.table = a.pages.table;
  p.num_pages = a.pages.num_pages;
  p.err = ctx->err;
  p.span = reinterpret_cast<int2*>(base + w.span);
  p.dropped = reinterpret_cast<int2*>(base + w.dropped);
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
  p.q_stage = (p.spread_s ? 16 : p.rows_s <= 32 ? 32 : 64) * 128;
  p.cost_pair = p.nbp * kCostPair + kCostPairSegment;
  const int single = p.spread_p && p.nbp >= kSpreadBlocks ? kCostSpread : p.rows_p <= 32 ? kCostFew : kCostSingle;
  p.cost_group = (p.npt - 1) * p.cost_pair + ((p.ntile & 1) ? p.nbp * single + kCostSegment : p.cost_pair);
  p.cost_prefix = p.Np > 0 ? p.cost_group * p.G : 0;
  p.scale_log2 = kLog2e / sqrtf(static_cast<float>(s.head_dim));
  // no more CTAs than blocks there can be
  const int64_t most = static_cast<int64_t>(p.nsp) * p.nbp + static_cast<int64_t>(p.B) * p.G * p.nb;
  const int grid =
      static_cast<int>(std::min<int64_t>(most, std::min(std::max(ctx->num_sms, 1), kMaxGrid)));
  p.grid = grid;
  return s.head_dim == 128 ? launch<128>(s, a, p, st) : launch<64>(s, a, p, st);
}

cudaError_t set_wait_limit_prefix(uint64_t ns) { return set_wait_limit_here(ns); }

}  // namespace msa
