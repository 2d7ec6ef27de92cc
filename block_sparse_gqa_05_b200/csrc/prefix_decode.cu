// Decode attention of a batch that shares a prefix, over own caches of
// different lengths, with the softmax weight each own key receives.
//
// Every query row (token, head) attends the prefix rows and the own rows it
// sees; one CTA per row, each of its warps over every fourth key with an
// online softmax (running maximum and sum, fp32), merged at the end.  The
// weights follow once the normalisers are known: a warp per own key computes
// its logits again and adds exp(s - lse) over the rows that see it.
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

struct PrefixParams {
  const uint16_t *q, *kp, *vp, *k, *v;
  uint16_t* o;
  float *lse, *lse_ws, *w_out;
  const float* w_in;
  const int32_t *lens, *prefix_pages, *table;
  uint32_t* err;
  int B, T, H, G, r, C, nb, Np, Cp, num_pages;
  float scale_log2;
};

// Valid rows of sequence b's own cache, clamped into [0, C].
__device__ __forceinline__ int own_len(const PrefixParams& p, int b) {
  const int n = p.lens[b];
  if (n >= 0 && n <= p.C) return n;
  atomicOr(p.err, kErrBadLength);
  return n < 0 ? 0 : p.C;
}

// Offset, in elements, of prefix row x of group g.
template <int D>
__device__ __forceinline__ long long prefix_row(const PrefixParams& p, int g, int x) {
  if (!p.prefix_pages) return (static_cast<long long>(g) * p.Cp + x) * D;
  const int pg = page_of(p.prefix_pages, 0, p.num_pages, 0, x >> 7, p.err);
  return ((static_cast<long long>(pg) * p.G + g) * 128 + (x & 127)) * D;
}

// Offset, in elements, of own row x of (b, g).
template <int D>
__device__ __forceinline__ long long own_row(const PrefixParams& p, int b, int g, int x) {
  if (!p.table) return ((static_cast<long long>(b) * p.G + g) * p.C + x) * D;
  const int pg = page_of(p.table, p.nb, p.num_pages, b, x >> 7, p.err);
  return ((static_cast<long long>(pg) * p.G + g) * 128 + (x & 127)) * D;
}

template <int D>
__device__ __forceinline__ void load_row(const uint16_t* src, int lane, float* out) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(src + i * 64 + 2 * lane);
    out[2 * i] = __uint_as_float(w << 16);
    out[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
}

template <int D>
__device__ __forceinline__ float dot_row(const float* a, const float* b) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) prefix_attn_kernel(const PrefixParams p) {
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = blockIdx.x;
  const int h = static_cast<int>(row % p.H), g = h / p.r;
  const int t = static_cast<int>(row / p.H % p.T), b = static_cast<int>(row / p.H / p.T);
  const int own = max(0, own_len(p, b) - p.T + t + 1);
  float q[D / 32], acc[D / 32], kv[D / 32];
  load_row<D>(p.q + row * D, lane, q);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int x = warp; x < p.Np + own; x += kWarps) {
    const bool pre = x < p.Np;
    const long long at = pre ? prefix_row<D>(p, g, x) : own_row<D>(p, b, g, x - p.Np);
    load_row<D>((pre ? p.kp : p.k) + at, lane, kv);
    const float s = dot_row<D>(q, kv) * p.scale_log2;
    const float mn = fmaxf(m, s);
    const float c = mn == -INFINITY ? 1.f : exp2f(m - mn);
    const float e = mn == -INFINITY ? 0.f : exp2f(s - mn);
    load_row<D>((pre ? p.vp : p.v) + at, lane, kv);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(acc[i], c, e * kv[i]);
    l = fmaf(l, c, e);
    m = mn;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    so[warp][i * 64 + 2 * lane] = acc[2 * i];
    so[warp][i * 64 + 2 * lane + 1] = acc[2 * i + 1];
  }
  __syncthreads();
  float M = -INFINITY, L = 0.f, O = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < kWarps; ++w) {
    const float c = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - M);
    L = fmaf(sl[w], c, L);
    if (threadIdx.x < D) O = fmaf(so[w][threadIdx.x], c, O);
  }
  if (threadIdx.x < D) {
    __nv_bfloat16 v = __float2bfloat16_rn(L > 0.f ? O / L : 0.f);
    p.o[row * D + threadIdx.x] = *reinterpret_cast<uint16_t*>(&v);
  }
  if (threadIdx.x == 0) {
    const float lse2 = L > 0.f ? M + log2f(L) : -INFINITY;
    if (p.lse_ws) p.lse_ws[row] = lse2;
    if (p.lse) p.lse[row] = lse2 / kLog2e;
  }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) prefix_weights_kernel(const PrefixParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bg = blockIdx.x, b = bg / p.G, g = bg % p.G;
  const int len = own_len(p, b);
  float kv[D / 32], q[D / 32];
  for (int x = blockIdx.y * kWarps + warp; x < len; x += gridDim.y * kWarps) {
    load_row<D>(p.k + own_row<D>(p, b, g, x), lane, kv);
    float w = 0.f;
    for (int t = max(0, x - (len - p.T)); t < p.T; ++t)
      for (int j = 0; j < p.r; ++j) {
        const long long row = (static_cast<long long>(b) * p.T + t) * p.H + g * p.r + j;
        load_row<D>(p.q + row * D, lane, q);
        const float s = dot_row<D>(q, kv) * p.scale_log2;
        w += exp2f(s - p.lse_ws[row]);
      }
    if (lane == 0) {
      const long long at = static_cast<long long>(bg) * p.C + x;
      p.w_out[at] = (p.w_in ? p.w_in[at] : 0.f) + w;
    }
  }
}

template <int D>
cudaError_t launch(const PrefixParams& p, cudaStream_t st) {
  {
    ProfScope ps_("prefix_attn", st);
    prefix_attn_kernel<D><<<static_cast<unsigned>(p.B) * p.T * p.H, kWarps * 32, 0, st>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.w_out) return e;
  {
    ProfScope ps_("prefix_weights", st);
    const dim3 grid(static_cast<unsigned>(p.B) * p.G,
                    static_cast<unsigned>(ceil_div(p.C, 64 * kWarps)));
    prefix_weights_kernel<D><<<grid, kWarps * 32, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

size_t prefix_decode_workspace_bytes(const msa_shape& s, bool weights) {
  (void)weights;
  return align_up(sizeof(float) * static_cast<size_t>(s.batch) * s.seq_q * s.n_q_heads, 256);
}

cudaError_t launch_prefix_decode(const msa_shape& s, const PrefixDecodeArgs& a, void* ws,
                                 cudaStream_t st) {
  const DevCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  PrefixParams p{};
  p.q = a.q;
  p.kp = a.prefix_pages ? a.k : a.kp;
  p.vp = a.prefix_pages ? a.v : a.vp;
  p.k = a.k;
  p.v = a.v;
  p.o = a.o;
  p.lse = a.lse;
  p.lse_ws = static_cast<float*>(ws);
  p.w_in = a.w_in;
  p.w_out = a.w_out;
  p.lens = a.lens;
  p.prefix_pages = a.prefix_pages;
  p.table = a.pages.table;
  p.num_pages = a.pages.num_pages;
  p.err = ctx->err;
  p.B = s.batch;
  p.T = s.seq_q;
  p.H = s.n_q_heads;
  p.G = s.n_kv_heads;
  p.r = s.n_q_heads / s.n_kv_heads;
  p.C = s.seq_kv;
  p.nb = static_cast<int>(ceil_div(s.seq_kv, 128));
  p.Np = a.prefix_len;
  p.Cp = a.prefix_cap;
  p.scale_log2 = kLog2e / sqrtf(static_cast<float>(s.head_dim));
  return s.head_dim == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace msa
