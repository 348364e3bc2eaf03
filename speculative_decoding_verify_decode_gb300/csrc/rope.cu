// The rotating append (include/sd_rope.h: sd_rope_append): q and k rows
// turned to their positions, k and v set into the paged bf16 cache on the way.
//
// y_a = x_a c - x_b s, y_b = x_b c + x_a s for every pair of the first rot_dim
// dims: 3 flops a value against 4 bytes, so bytes are all there is, and each
// row is read once and written once to each place it goes to.
//
// One CTA a row.  Its positions' cosines and sines serve every head: they are
// loaded once into shared memory (a load per head would ask L1 for as many bytes
// again as the heads themselves).  A thread turns eight pairs, two 16-byte pieces half a
// rotation apart (or, interleaved, one piece of four pairs); the row's own pieces
// are asked for before the table's are waited for, so a row costs one latency.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace sdv {
namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float2 pair_value(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ uint32_t pair_bits(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The dims of a piece against those of its mate.
__device__ __forceinline__ void turn(uint4& a, uint4& b, const float* c, const float* s) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
  uint32_t* y = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = pair_value(x[i]), v = pair_value(y[i]);
    const float2 cc = *reinterpret_cast<const float2*>(c + 2 * i), ss = *reinterpret_cast<const float2*>(s + 2 * i);
    x[i] = pair_bits(u.x * cc.x - v.x * ss.x, u.y * cc.y - v.y * ss.y);
    y[i] = pair_bits(v.x * cc.x + u.x * ss.x, v.y * cc.y + u.y * ss.y);
  }
}
// Neighbouring dims against each other: four pairs of one piece.
__device__ __forceinline__ void turn(uint4& a, const float* c, const float* s) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
  const float4 cc = *reinterpret_cast<const float4*>(c), ss = *reinterpret_cast<const float4*>(s);
  const float* cf = &cc.x;
  const float* sf = &ss.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = pair_value(x[i]);
    x[i] = pair_bits(u.x * cf[i] - u.y * sf[i], u.y * cf[i] + u.x * sf[i]);
  }
}

template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_append_kernel(const RopeParams p) {
  __shared__ __align__(16) float s_table[SD_ROPE_MAX_DIM];
  const int row = blockIdx.x, t = threadIdx.x;
  pdl_wait();
  const int pos = p.positions[row];
  int slot = p.slots != nullptr ? p.slots[row] : -1;
  if (pos < 0 || pos >= p.table_len) {
    if (pos != -1 && t == 0) report(p.dev_status, SD_DEV_BAD_POSITION);
    return;
  }
  if (slot < -1 || slot / kPage >= p.num_pool_pages) {
    if (t == 0) report(p.dev_status, SD_DEV_BAD_SLOT);
    slot = -1;
  }
  // Items of a rotated head: `turned` pairs of pieces (or single pieces), then `plain` pieces behind rot_dim; then V's.
  const int half = p.rot_dim / 2;
  const int turned = INTER ? p.rot_dim / 8 : p.rot_dim / 16, plain = (p.dim - p.rot_dim) / 8, per_head = turned + plain;
  const int heads = p.hq + p.hkv, rotated = heads * per_head;
  const int items = rotated + (slot >= 0 ? p.hkv * (p.dim / 8) : 0);
  const size_t page = slot >= 0 ? (size_t)(slot / kPage) * p.hkv : 0;
  const int in_page = slot >= 0 ? slot % kPage : 0;
  const float inv = 1.0f / (float)per_head, inv_v = 8.0f / (float)p.dim;

  struct Item {
    uint4 a, b;
    const float* c;              // null: not turned
    __nv_bfloat16 *out, *cache;  // where the first piece goes (nullable)
    int mate;                    // dims from the first piece to the second, 0: none
  };
  auto fetch = [&](int i) {
    Item it;
    it.c = nullptr;
    it.out = it.cache = nullptr;
    it.mate = 0;
    it.a = it.b = make_uint4(0, 0, 0, 0);
    if (i >= items) return it;
    const bool is_v = i >= rotated;
    // quotients by one multiplication: exact, the halves keep them away from the borders (i < 2^17)
    const int j = is_v ? i - rotated : i;
    const int per = is_v ? p.dim / 8 : per_head;
    const int h = __float2int_rz(((float)j + 0.5f) * (is_v ? inv_v : inv)), e = j - h * per;
    int d;
    if (is_v) d = e * 8;
    else if (e < turned) d = e * 8;
    else d = p.rot_dim + (e - turned) * 8;
    const __nv_bfloat16* src;
    if (is_v) {
      src = p.v + (long long)row * p.v_stride + h * p.dim + d;
    } else if (h < p.hq) {
      src = p.q + (long long)row * p.q_stride + h * p.dim + d;
      it.out = p.q_out + (long long)row * p.q_out_stride + h * p.dim + d;
    } else {
      src = p.k + (long long)row * p.k_stride + (h - p.hq) * p.dim + d;
      if (p.k_out != nullptr) it.out = p.k_out + (long long)row * p.k_out_stride + (h - p.hq) * p.dim + d;
    }
    if (slot >= 0 && (is_v || h >= p.hq))
      it.cache = (is_v ? p.v_cache : p.k_cache) + ((page + (is_v ? h : h - p.hq)) * kPage + in_page) * p.dim + d;
    it.a = *reinterpret_cast<const uint4*>(src);
    if (!is_v && e < turned) {
      it.c = s_table + (INTER ? e * 4 : e * 8);
      if (!INTER) {
        it.mate = half;
        it.b = *reinterpret_cast<const uint4*>(src + half);
      }
    }
    return it;
  };
  auto finish = [&](Item& it) {
    if (it.c != nullptr) {
      if (INTER) turn(it.a, it.c, it.c + half);
      else turn(it.a, it.b, it.c, it.c + half);
    }
    if (it.out != nullptr) {
      *reinterpret_cast<uint4*>(it.out) = it.a;
      if (it.mate) *reinterpret_cast<uint4*>(it.out + it.mate) = it.b;
    }
    if (it.cache != nullptr) {
      *reinterpret_cast<uint4*>(it.cache) = it.a;
      if (it.mate) *reinterpret_cast<uint4*>(it.cache + it.mate) = it.b;
    }
  };
  Item x = fetch(t), y = fetch(t + kRopeThreads);
  for (int i = t; i < p.rot_dim / 4; i += kRopeThreads)
    reinterpret_cast<float4*>(s_table)[i] = __ldg(reinterpret_cast<const float4*>(p.table + (size_t)pos * p.rot_dim) + i);
  __syncthreads();
  finish(x);
  finish(y);
  for (int i = t + 2 * kRopeThreads; i < items; i += 2 * kRopeThreads) {
    x = fetch(i);
    y = fetch(i + kRopeThreads);
    finish(x);
    finish(y);
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, cudaStream_t st) {
  if (p.num_rows == 0 || p.hq + p.hkv == 0) return cudaSuccess;
  return p.interleaved ? launch_pdl(rope_append_kernel<true>, dim3(p.num_rows), dim3(kRopeThreads), 0, st, p)
                       : launch_pdl(rope_append_kernel<false>, dim3(p.num_rows), dim3(kRopeThreads), 0, st, p);
}

}  // namespace sdv
