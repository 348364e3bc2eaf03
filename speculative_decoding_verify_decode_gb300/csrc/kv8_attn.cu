// Verify attention over the 8-bit block-scaled cache (include/sd_kv8.h:
// sd_kv8_attn), the plain kernel: one CTA per (node row, query head), one warp
// per key at a time, fp32 throughout, one pass with each warp's running
// maximum and sum, the eight warps joined at the end.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace sdv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float2 e4m3x2_value(uint32_t codes) {
  uint32_t h;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"(codes & 0xffffu));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv8_attn_plain_kernel(const Kv8AttnParams p, const BatchDesc bd) {
  constexpr int E = D / 32;   // values per lane
  const int r = blockIdx.x, h = blockIdx.y, g = h / (p.hq / p.hkv);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int b = 0, hi = bd.batch - 1;
  while (b < hi) {
    const int mid = (b + hi + 1) >> 1;
    if (bd.q_indptr[mid] <= r) b = mid; else hi = mid - 1;
  }
  const int q0 = bd.q_indptr[b], node = r - q0;
  int L = p.ctx_lens[b];
  if (L < 0 || L > p.max_pages * kPage) {
    if (threadIdx.x == 0) report(p.dev_status, SD_DEV_BAD_CTX);
    L = L < 0 ? 0 : p.max_pages * kPage;
  }
  // the root path
  unsigned long long see = 1ull << node;
  int depth = 0;
  for (int u = node; u >= 0;) {
    const int up = p.parents[q0 + u];
    if (u == 0 ? up != -1 : (up < 0 || up >= u)) {
      if (threadIdx.x == 0) report(p.dev_status, SD_DEV_BAD_PARENTS);
      see = 1ull << node;
      depth = 0;
      break;
    }
    if (u == 0) break;
    see |= 1ull << up;
    ++depth;
    u = up;
  }
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[(long long)r * p.q_stride + h * D + lane * E + e]) * p.scale;
    acc[e] = 0.f;
  }
  const float slope = p.slopes != nullptr ? p.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f;
  auto take = [&](const float (&k)[E], const float (&v)[E], int away) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (p.softcap > 0.f) s = p.softcap * tanhf(s / p.softcap);
    if (p.slopes != nullptr) s += slope * (float)away;
    const float mn = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.f : expf(m - mn), w = expf(s - mn);
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * v[e];
    m = mn;
  };
  const int q_pos = L + depth;
  const int t_first = p.window > 0 ? max(0, q_pos - p.window + 1) : 0;
  for (int t = t_first + warp; t < L; t += kThreads / 32) {
    const int page = p.page_table[(size_t)b * p.max_pages + t / kPage];
    float k[E], v[E];
    if (page < 0 || page >= p.num_pool_pages) {
      report(p.dev_status, SD_DEV_BAD_PAGE);
#pragma unroll
      for (int e = 0; e < E; ++e) k[e] = v[e] = 0.f;
    } else {
      const size_t block = (size_t)page * p.hkv + g;
      float sk = p.k_scales[block], sv = p.v_scales[block];
      const float lo = 0x1p-100f, up = 0x1p100f;
      if (!(sk >= lo && sk <= up) || !(sv >= lo && sv <= up)) {
        report(p.dev_status, SD_DEV_BAD_SCALE);
        sk = fminf(fmaxf(sk, lo), up);
        sv = fminf(fmaxf(sv, lo), up);
      }
      const size_t at = (block * kPage + t % kPage) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 a = e4m3x2_value(*reinterpret_cast<const uint16_t*>(p.k_cache + at + e));
        const float2 c = e4m3x2_value(*reinterpret_cast<const uint16_t*>(p.v_cache + at + e));
        k[e] = a.x * sk; k[e + 1] = a.y * sk;
        v[e] = c.x * sv; v[e + 1] = c.y * sv;
      }
    }
    take(k, v, t - q_pos);
  }
  int up = depth;   // the path's nodes from the deepest: depth of the next one
  if (warp == 0) {
    for (int n = node; n >= 0; --n) {
      if (!((see >> n) & 1ull)) continue;
      const int away = up - depth;
      --up;
      if (p.window > 0 && away <= -p.window) continue;
      float k[E], v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = __bfloat162float(p.k_new[(long long)(q0 + n) * p.k_stride + g * D + lane * E + e]);
        v[e] = __bfloat162float(p.v_new[(long long)(q0 + n) * p.v_stride + g * D + lane * E + e]);
      }
      take(k, v, away);
    }
  }
  __shared__ float s_m[kThreads / 32], s_l[kThreads / 32], s_acc[kThreads / 32][D];
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
  __syncthreads();
  float mm = s_m[0];
  for (int w = 1; w < kThreads / 32; ++w) mm = fmaxf(mm, s_m[w]);
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float sum = 0.f, den = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (s_m[w] == -INFINITY) continue;
      const float f = expf(s_m[w] - mm);
      sum += f * s_acc[w][d];
      den += f * s_l[w];
    }
    p.out[((size_t)r * p.hq + h) * D + d] = __float2bfloat16_rn(sum / den);
    if (p.lse != nullptr && d == 0) p.lse[(size_t)r * p.hq + h] = mm + logf(den);
  }
}

}  // namespace

size_t kv8_attn_workspace(int, int, int, const BatchDesc&) { return 0; }

cudaError_t launch_kv8_attn(const Kv8AttnParams& p, const BatchDesc& bd, cudaStream_t st) {
  const dim3 grid(bd.total_nodes, p.hq);
  if (p.dim == 256)
    kv8_attn_plain_kernel<256><<<grid, kThreads, 0, st>>>(p, bd);
  else
    kv8_attn_plain_kernel<128><<<grid, kThreads, 0, st>>>(p, bd);
  return cudaGetLastError();
}

}  // namespace sdv
