// The rotating append (include/sd_rope.h: sd_rope_append): q and k rows
// turned to their positions, k and v set into the paged bf16 cache on the way.
//
// y_a = x_a c - x_b s, y_b = x_b c + x_a s for every pair of the first rot_dim
// dims: 3 flops a value against 4 bytes, so bytes are all there is, and each
// row is read once and written once to each place it goes to.
//
// One CTA a row.  Its positions' cosines and sines serve every head: they are
// loaded once into shared memory (a load per head would ask L1 for as many bytes
// again as the heads themselves).  An item is two 16-byte pieces of a head, half the turning or half the
// other dims apart: eight pairs that turn (or, interleaved, twice four), or sixteen values that do not.  A thread has
// two of them, asked for before the row's position and its table are waited for, so a row costs one latency,
// and the six rows of an SM hide it: 8191 rows of 24 + 4 + 4 heads of 256 dims, 64 of them turning, 42 us, 0.94 of the copy
// rate (four rows 50, five 46.5, eight 42.6; all 256 turning 48 us).  One row alone is bound by latency: 2.7 us for 40.
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
__global__ void __launch_bounds__(kRopeThreads, 6) rope_append_kernel(const RopeParams p) {
  __shared__ __align__(16) float s_table[SD_ROPE_MAX_DIM];
  const int row = blockIdx.x, t = threadIdx.x;
  pdl_wait();
  const int pos = p.positions[row];
  int slot = p.slots != nullptr ? p.slots[row] : -1;
  const int half = p.rot_dim / 2, other = (p.dim - p.rot_dim) / 2;
  const int turned = p.rot_dim / 16, per_head = p.dim / 16;      // items of a head
  const int heads = p.hq + p.hkv + (p.v != nullptr ? p.hkv : 0), items = heads * per_head;
  const float inv = 1.0f / (float)per_head;
  // An item's head (V's behind the others), first dim and the distance of its second piece; the quotient by one
  // multiplication: exact, the half keeps it away from the borders (i < 2^17).
  auto place = [&](int i, int& h, int& d, int& mate) {
    h = __float2int_rz(((float)i + 0.5f) * inv);
    const int e = i - h * per_head;
    const bool is_v = h >= p.hq + p.hkv, turns = !is_v && e < turned;
    d = is_v || turns ? e * 8 : p.rot_dim + (e - turned) * 8;
    mate = is_v ? p.dim / 2 : turns ? half : other;
    return turns;
  };
  auto fetch = [&](int i, uint4& a, uint4& b) {
    if (i >= items) return;
    int h, d, mate;
    place(i, h, d, mate);
    const __nv_bfloat16* src = h < p.hq              ? p.q + (long long)row * p.q_stride + h * p.dim
                               : h < p.hq + p.hkv    ? p.k + (long long)row * p.k_stride + (h - p.hq) * p.dim
                                                     : p.v + (long long)row * p.v_stride + (h - p.hq - p.hkv) * p.dim;
    a = *reinterpret_cast<const uint4*>(src + d);
    b = *reinterpret_cast<const uint4*>(src + d + mate);
  };
  auto finish = [&](int i, uint4& a, uint4& b) {
    if (i >= items) return;
    int h, d, mate;
    if (place(i, h, d, mate)) {
      if (INTER) {
        turn(a, s_table + d / 2, s_table + d / 2 + half);
        turn(b, s_table + (d + half) / 2, s_table + (d + half) / 2 + half);
      } else {
        turn(a, b, s_table + d, s_table + d + half);
      }
    }
    __nv_bfloat16* out = nullptr;
    if (h < p.hq) out = p.q_out + (long long)row * p.q_out_stride + h * p.dim + d;
    else if (h < p.hq + p.hkv && p.k_out != nullptr) out = p.k_out + (long long)row * p.k_out_stride + (h - p.hq) * p.dim + d;
    if (out != nullptr) {
      *reinterpret_cast<uint4*>(out) = a;
      *reinterpret_cast<uint4*>(out + mate) = b;
    }
    if (h >= p.hq && slot >= 0) {
      const bool is_v = h >= p.hq + p.hkv;
      __nv_bfloat16* cache = (is_v ? p.v_cache : p.k_cache) +
                             (((size_t)(slot / kPage) * p.hkv + (h - p.hq - (is_v ? p.hkv : 0))) * kPage + slot % kPage) * p.dim + d;
      *reinterpret_cast<uint4*>(cache) = a;
      *reinterpret_cast<uint4*>(cache + mate) = b;
    }
  };
  // the row's own pieces are asked for before its position is known
  constexpr int U = 2;
  uint4 a[U], b[U];
#pragma unroll
  for (int k = 0; k < U; ++k) fetch(t + k * kRopeThreads, a[k], b[k]);
  if (pos < 0 || pos >= p.table_len) {
    if (pos != -1 && t == 0) report(p.dev_status, SD_DEV_BAD_POSITION);
    return;
  }
  if (slot < -1 || slot / kPage >= p.num_pool_pages) {
    if (t == 0 && p.slots != nullptr) report(p.dev_status, SD_DEV_BAD_SLOT);
    slot = -1;
  }
  for (int i = t; i < p.rot_dim / 4; i += kRopeThreads)
    reinterpret_cast<float4*>(s_table)[i] = __ldg(reinterpret_cast<const float4*>(p.table + (size_t)pos * p.rot_dim) + i);
  __syncthreads();
#pragma unroll 1
  for (int i = t;;) {
#pragma unroll
    for (int k = 0; k < U; ++k) finish(i + k * kRopeThreads, a[k], b[k]);
    i += U * kRopeThreads;
    if (i - t >= items) break;
#pragma unroll
    for (int k = 0; k < U; ++k) fetch(i + k * kRopeThreads, a[k], b[k]);
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, cudaStream_t st) {
  if (p.num_rows == 0 || p.hq + p.hkv == 0) return cudaSuccess;
  return p.interleaved ? launch_pdl(rope_append_kernel<true>, dim3(p.num_rows), dim3(kRopeThreads), 0, st, p)
                       : launch_pdl(rope_append_kernel<false>, dim3(p.num_rows), dim3(kRopeThreads), 0, st, p);
}

}  // namespace sdv
