// Quantising append into the 8-bit block-scaled cache (include/sd_kv8.h:
// sd_kv8_append).
//
// Per (layer, K or V, page, KV head): amax of the new rows, the smallest
// power of two s with amax <= 448 s, the larger of it and the page's old
// scale, and code = e4m3(x / s).  A power of two costs an e4m3 value nothing
// (its relative precision does not depend on where in the exponent range it
// lies) and makes x / s and the move of old codes to a grown scale exact but
// for the final rounding.
//
// The pass is bound by HBM: 4 bytes read and 2 written per (K, V) value pair.
// One warp owns one (layer, tensor, head, page): it holds the page's new rows
// (up to 16 x head_dim bf16, at most 64 registers a lane) so that amax and
// quantisation read them once, with all their 16-byte loads in flight; lanes
// own 8 consecutive values, so a row is read in 16-byte and written in 8-byte
// pieces, coalesced.  No atomics: a page's rows are consecutive in the slot
// map, the first of them names the owner.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace sdv {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kMinExp = SD_KV8_MIN_SCALE_EXP, kMaxExp = SD_KV8_MAX_SCALE_EXP;

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// Two fp32 values as two e4m3 codes (lo in the low byte), nearest-even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{ .reg .b16 t; cvt.rn.satfinite.e4m3x2.f32 t, %1, %2; cvt.u32.u16 %0, t; }" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t codes) {
  uint32_t h;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"(codes & 0xffffu));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 bf16x2_value(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// Four bf16 (two words) as four codes: x * inv when 1 / scale is exact (a power of two), else x / scale.
__device__ __forceinline__ uint32_t quantise4(uint32_t a, uint32_t b, float scale, float inv, bool exact) {
  const float2 x = bf16x2_value(a), y = bf16x2_value(b);
  if (exact) return e4m3x2(x.x * inv, x.y * inv) | (e4m3x2(y.x * inv, y.y * inv) << 16);
  return e4m3x2(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale)) |
         (e4m3x2(__fdiv_rn(y.x, scale), __fdiv_rn(y.y, scale)) << 16);
}
__device__ __forceinline__ uint32_t requantise4(uint32_t c, float ratio) {
  const float2 x = e4m3x2_value(c), y = e4m3x2_value(c >> 16);
  return e4m3x2(x.x * ratio, x.y * ratio) | (e4m3x2(y.x * ratio, y.y * ratio) << 16);
}

// D: head_dim.  A CTA looks at `window` rows of the slot map; each row that
// begins a page there gives 2 * heads warp tasks.
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 6) kv8_append_kernel(const Kv8AppendParams p, const int window) {
  constexpr int kLanes = D / 8;            // lanes per row (8 values each)
  constexpr int kRowsAtOnce = 32 / kLanes; // rows a warp touches per step
  constexpr int kSteps = kPage / kRowsAtOnce;
  __shared__ int s_lead[kPage], s_n;
  const int layer = blockIdx.y;
  const int r_base = blockIdx.x * window;
  if (threadIdx.x < 32) {
    const int t = threadIdx.x, r = r_base + t;
    bool lead = false;
    if (t < window && r < p.max_rows) {
      const int slot = p.slots[r], prev = r > 0 ? p.slots[r - 1] : -1;
      if (slot < -1 || slot / kPage >= p.num_pool_pages) {
        if (layer == 0) report(p.dev_status, SD_DEV_BAD_SLOT);
      } else if (slot >= 0) {
        lead = prev < 0 || prev / kPage != slot / kPage;
      }
    }
    const uint32_t m = __ballot_sync(0xffffffffu, lead);
    if (lead) s_lead[__popc(m & ((1u << t) - 1u))] = r;
    if (t == 0) s_n = __popc(m);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int combos = 2 * p.heads;
  const int col = lane % kLanes, sub = lane / kLanes;
  for (int task = blockIdx.z * (kAppendThreads / 32) + warp; task < s_n * combos; task += gridDim.z * (kAppendThreads / 32)) {
    const int r0 = s_lead[task / combos], combo = task % combos;
    const int head = combo >> 1;
    const bool is_v = combo & 1;
    // the group: the following rows on the same page, which must rise by one (a seventeenth cannot)
    const int slot0 = p.slots[r0], page = slot0 / kPage, first = slot0 % kPage;
    int slot = -1, src = -1;
    if (lane <= kPage && r0 + lane < p.max_rows) {
      slot = p.slots[r0 + lane];
      src = p.rows != nullptr ? p.rows[r0 + lane] : r0 + lane;
    }
    const bool same = lane <= kPage && slot >= 0 && slot / kPage == page;
    const int n = __ffs(~__ballot_sync(0xffffffffu, same)) - 1;   // 1..17
    const bool wrong = lane < n && (slot != slot0 + lane || src < 0 || src >= p.num_src_rows);
    if (__any_sync(0xffffffffu, wrong)) {
      if (lane == 0 && layer == 0) report(p.dev_status, SD_DEV_BAD_SLOT);
      continue;
    }
    const __nv_bfloat16* x = (is_v ? p.v_new[layer] : p.k_new[layer]) + head * D + col * 8;
    uint4 v[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = k * kRowsAtOnce + sub;
      const int from = __shfl_sync(0xffffffffu, src, i);
      v[k] = make_uint4(0, 0, 0, 0);
      if (i < n) v[k] = __ldg(reinterpret_cast<const uint4*>(x + (long long)from * p.new_stride));
    }
    const size_t block = (size_t)page * p.heads + head;
    float* scale_at = (is_v ? p.v_scale[layer] : p.k_scale[layer]) + block;
    uint8_t* codes = (is_v ? p.v_cache[layer] : p.k_cache[layer]) + block * (kPage * D) + col * 8;
    const float old = first > 0 ? *scale_at : 0.f;
    if (first > 0 && !(old >= pow2i(kMinExp) && old <= pow2i(kMaxExp))) {
      if (lane == 0) report(p.dev_status, SD_DEV_BAD_SCALE);
      continue;
    }
    // amax as bf16 bits: magnitudes order like integers; infinities and NaN sort above every finite value
    uint32_t am = 0;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      am = __vmaxu2(am, __vmaxu2(__vmaxu2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu),
                                 __vmaxu2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu)));
    }
    uint32_t a = max(am & 0xffffu, am >> 16);
    a = __reduce_max_sync(0xffffffffu, a);
    if (a >= 0x7f80u) {   // rare: take the finite values alone
      a = 0;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
          a = max(a, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
      }
      a = __reduce_max_sync(0xffffffffu, a);
    }
    // 448 * 2^e = 1.75 * 2^(e + 8): the exponent of amax less 8, one more when its mantissa is above 1.75
    const int e = min(kMaxExp, max(kMinExp, (int)(a >> 7) - 127 - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0)));
    const float scale = fmaxf(old, pow2i(e));
    if (first > 0 && scale != old) {
      const float ratio = old / scale;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int i = k * kRowsAtOnce + sub;
        if (i < first) {
          uint2* at = reinterpret_cast<uint2*>(codes + i * D);
          const uint2 c = *at;
          *at = make_uint2(requantise4(c.x, ratio), requantise4(c.y, ratio));
        }
      }
    }
    const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0u;
    const float inv = 1.f / scale;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = k * kRowsAtOnce + sub;
      if (i < n)
        *reinterpret_cast<uint2*>(codes + (first + i) * D) =
            make_uint2(quantise4(v[k].x, v[k].y, scale, inv, exact), quantise4(v[k].z, v[k].w, scale, inv, exact));
    }
    if (lane == 0 && scale != old) *scale_at = scale;
  }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendParams& p, cudaStream_t st) {
  if (p.max_rows == 0) return cudaSuccess;
  // Rows per CTA: a row of its own while that fills the machine about twice over at most (single tokens of a batch, an
  // accepted path: 6 tokens in 16 layers 3.7 us, against 5.5 by sixteens); for prompts sixteen, of which one begins a page
  // (8191 tokens 11.0 us, against 20.3 by single rows).  11.0 us are 4.6 TB/s of the pass's 50 MB.
  const int window = (long long)p.max_rows * p.num_layers <= 4 * kSMs ? 1 : kPage;
  // enough CTAs per window for one page's tasks, a warp each, four to a CTA (eight: 11.4 us and 3.9 for the same two)
  const int share = (2 * p.heads + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  const dim3 grid((p.max_rows + window - 1) / window, p.num_layers, share);
  if (p.dim == 256)
    kv8_append_kernel<256><<<grid, kAppendThreads, 0, st>>>(p, window);
  else
    kv8_append_kernel<128><<<grid, kAppendThreads, 0, st>>>(p, window);
  return cudaGetLastError();
}

}  // namespace sdv
