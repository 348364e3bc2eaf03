// The launch of attentions whose line of units is cut over the SMs (the 8-bit
// and the 4-bit cache): the SM count, the workspace's parts, and the merge of
// split segments.  P is the attention's parameter block.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace sdv {
namespace {

inline int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    cudaGetLastError();   // no device here
    return kSMs;
  }
  return sms;
}

// Log-sum-exp merge of the segments that piece borders cut: o = sum 2^(lse_s - M) o_s / sum 2^(lse_s - M).
// One block per (node row, query head): four warps each take every fourth partial, a lane D / 32 dims, with the
// loads of kBatch partials in flight per warp (40 partials in one round of latency).
constexpr int kMergeThreads = 128, kMergeWarps = 4, kBatch = 10;

template <int D, typename P>
__global__ void __launch_bounds__(kMergeThreads) kv_merge_kernel(const P p, const BatchDesc bd) {
  constexpr int E = D / 32;   // dims per lane
  const int r = blockIdx.x, h = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int b = 0, hi = bd.batch - 1;
  while (b < hi) {
    const int mid = (b + hi + 1) >> 1;
    if (bd.q_indptr[mid] <= r) b = mid; else hi = mid - 1;
  }
  const int g = h / p.group, c = (h % p.group) / p.hpc, part0 = c * p.hpc;
  const int hpc = min(p.hpc, p.group - part0);
  const int col = (r - bd.q_indptr[b]) * hpc + h % p.group - part0;
  const int parts = p.hkv * p.hparts, s = g * p.hparts + c;
  int L = p.ctx_lens[b];
  L = L < 0 ? 0 : min(L, p.max_pages * kPage);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the attention kernel's partials and unit sums
  const int per = p.cum[kMaxBatch + 1], extra = p.cum[kMaxBatch + 2];
  const int cum = p.cum[b], line = (p.cum[b + 1] - cum) / parts;
  const int units = extra < 0 ? line : 1 + extra + (L - window_base(L, p.window, kTileTokens) + kTileTokens - 1) / kTileTokens;
  const int u0 = cum + s * line, k0 = u0 / per, n = (u0 + units - 1) / per - k0 + 1;
  if (n == 1) return;   // written directly
  const size_t slot0 = (size_t)k0 + b * parts + s;
  float mx = -INFINITY, den = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int base = warp; base < n; base += kMergeWarps * kBatch) {
    float w[kBatch];
    float o[kBatch][E];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + k * kMergeWarps;
      const size_t at = (slot0 + min(i, n - 1)) * p.nq + col;
      w[k] = i < n ? p.lse_part[at] : -INFINITY;
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(&o[k][e]) = *reinterpret_cast<const float4*>(p.o_part + at * D + lane * E + e);
    }
    float bm = mx;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) bm = fmaxf(bm, w[k]);
    const float a = mx == -INFINITY ? 0.f : fast_exp2(mx - bm);
    den *= a;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= a;
    mx = bm;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (w[k] == -INFINITY) continue;                   // nothing visible there, or padding (a NaN goes on)
      const float f = fast_exp2(w[k] - mx);
      den += f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += f * o[k][e];
    }
  }
  // Every load is under way or done: the next kernel's blocks may come as this one's leave (at the start of the block
  // they took the SMs of a large merge: 512 rows of 16 partials 209 -> 224 us for the whole call).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float s_m[kMergeWarps], s_d[kMergeWarps], s_acc[kMergeWarps][D];
  if (lane == 0) { s_m[warp] = mx; s_d[warp] = den; }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
  __syncthreads();
  float m = s_m[0];
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) m = fmaxf(m, s_m[w]);
  float f[kMergeWarps], d = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    f[w] = s_m[w] == -INFINITY && s_d[w] == 0.f ? 0.f : fast_exp2(s_m[w] - m);
    d += f[w] * s_d[w];
  }
  const float inv = 1.f / d;
  constexpr int T = D / 2;    // threads that write a pair of dims
  if (threadIdx.x < T) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      const float2 v = *reinterpret_cast<const float2*>(&s_acc[w][2 * threadIdx.x]);
      x += f[w] * v.x;
      y += f[w] * v.y;
    }
    *reinterpret_cast<__nv_bfloat162*>(p.out + ((size_t)r * p.hq + h) * D + 2 * threadIdx.x) =
        __floats2bfloat162_rn(x * inv, y * inv);
  }
  if (p.lse != nullptr && threadIdx.x == 0) p.lse[(size_t)r * p.hq + h] = (m + fast_log2(d)) * kLn2;
}

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct Layout {
  size_t o, lse, total;   // cum at 0
};
// nq columns a piece, `ctas` CTAs per SM, hparts head parts of a KV group.
inline Layout layout_of(int nq, int ctas, int hparts, int hkv, int dim, const BatchDesc& bd, int sms) {
  // a piece and a segment name a partial; along the line of units their numbers rise together
  const size_t slots = (size_t)sms * ctas + (size_t)bd.batch * hkv * hparts;
  Layout l;
  l.o = align_up((kMaxBatch + 3) * sizeof(int));
  l.lse = l.o + align_up(slots * nq * dim * sizeof(float));
  l.total = l.lse + align_up(slots * nq * sizeof(float));
  return l;
}

}  // namespace
}  // namespace sdv
