// Quantising append into the 4-bit cache, and rows read back out of it
// (include/sd_kv4.h: sd_kv4_append, sd_kv4_read).
//
// Append.  Per block of 32 dims of a row: m, the value largest in magnitude;
// s = m / -8 in 5 bits; c = rint(x / s) + 8.  x / s is a quotient of an 8-bit and a
// 5-bit number, so it is either exactly half way between two integers or at
// least 2^-13 away from that: the product with an approximate reciprocal (off by 2^-20 at most), rounded to a
// multiple of 2^-16, is right in both cases, and no division is needed.  Two values share each step: the maxima are of
// 16-bit pairs, the roundings of fp32 pairs.
//
// One warp owns one (layer, K or V, page, KV head): the page's new rows are
// in its registers, so bytes are read once, and V's words, which hold eight
// tokens each, are put together without a second writer.  A lane has eight
// consecutive dims: four lanes are a block, two shuffles its maximum.  K's words go through
// shared memory (a row's lie 256 bytes apart), so that both records leave in
// 16-byte pieces.  Bound by HBM: 2 bytes read and 9/16 written a value.
//
// Read.  One warp per (layer, K or V, KV head, up to 16 entries of the slot map); V's
// words of a page are loaded once for the entries that lie on it.
#include "kernels.h"
#include "kv4_format.cuh"

namespace sdv {
namespace {

constexpr int kRowsThreads = 128, kRowsWarps = kRowsThreads / 32;

// The largest finite magnitude of eight bf16 values, as a key: magnitude, then the earlier index, then the sign.
__device__ __forceinline__ uint32_t top_key(const uint4 x, int index0) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t key = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
    const uint32_t mag = b & 0x7fffu;
    const uint32_t k = mag << 6 | (uint32_t)(31 - (index0 + e)) << 1 | b >> 15;
    key = max(key, mag < 0x7f80u ? k : 0u);
  }
  return key;
}
// bf16 bits of the block's scale: m / -8 with 5 significant bits, ties to even.
__device__ __forceinline__ uint32_t scale_of(uint32_t key) {
  const uint32_t mag = key >> 6, sign = key & 1u;
  if (mag < (27u << 7)) return 0u;                                     // below 2^-100
  const uint32_t r = (mag + 3u + ((mag >> 3) & 1u)) & 0x7ff8u;
  return min(r - (3u << 7), kKv4BadScale - 8u) | (sign ^ 1u) << 15;
}
__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// Infinities become the block's largest magnitude, NaN zero.
__device__ __forceinline__ uint32_t tamed(uint32_t two, uint32_t mag) {
  uint32_t r = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b = two >> (16 * h) & 0xffffu;
    if ((b & 0x7fffu) == 0x7f80u) b = (b & 0x8000u) | mag;
    else if ((b & 0x7fffu) > 0x7f80u) b = 0u;
    r |= b << (16 * h);
  }
  return r;
}
// Magnitudes beyond 8 times the largest scale become the largest that it reaches.
__device__ __forceinline__ uint32_t reached(uint32_t two) {
  const uint32_t top = kKv4BadScale - 8u + (3u << 7);     // 8 * 1.3125 * 2^123
  return (two & 0x80008000u) | __vminu2(two & 0x7fff7fffu, top | top << 16);
}
__device__ __forceinline__ bool wild(const uint4 x) {   // a NaN or an infinity among eight
  const uint32_t e = 0x7f807f80u;
  return (__vcmpeq2(x.x & e, e) | __vcmpeq2(x.y & e, e) | __vcmpeq2(x.z & e, e) | __vcmpeq2(x.w & e, e)) != 0u;
}

// Codes of a pair of values, one in each half.  inv: 1 / s (0 for s = 0: both codes are 8).  200 + q has multiples of
// 2^-16, which leaves a tie one; that plus 2^23 - 192 is 2^23 + (q + 8) rounded to even.  |q| <= 8.25, so what there is to
// keep within 0..15 is 16.
__device__ __forceinline__ uint32_t codes2(uint32_t two, float inv) {
  const float2 x = make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
  uint64_t q, c;
  const float2 k200 = make_float2(200.f, 200.f), k23 = make_float2(8388416.f, 8388416.f), f = make_float2(inv, inv);
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(*reinterpret_cast<const uint64_t*>(&x)),
      "l"(*reinterpret_cast<const uint64_t*>(&f)), "l"(*reinterpret_cast<const uint64_t*>(&k200)));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(q), "l"(*reinterpret_cast<const uint64_t*>(&k23)));
  return __vminu2(__byte_perm((uint32_t)c, (uint32_t)(c >> 32), 0x5410), 0x000f000fu);
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads, 4) kv4_append_kernel(const Kv4RowsParams p, const int window) {
  constexpr int kLanes = D / 8;            // lanes per row (8 values each)
  constexpr int kRowsAtOnce = 32 / kLanes; // rows a warp touches per step
  constexpr int kSteps = kPage / kRowsAtOnce;
  constexpr int kBlocks = D / kKv4Block;
  __shared__ int s_lead[kPage], s_n;
  __shared__ __align__(16) uint32_t s_k[kRowsWarps][kPage * D / 8];
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
#pragma unroll 1
  for (int task = blockIdx.z * kRowsWarps + warp; task < s_n * combos; task += gridDim.z * kRowsWarps) {
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
    const __nv_bfloat16* x = (is_v ? p.v_rows[layer] : p.k_rows[layer]) + head * D + col * 8;
    // A lane's rows by their token in the page: step k is token k * kRowsAtOnce + sub.
    uint4 v[kSteps];
    bool any_wild = false;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = k * kRowsAtOnce + sub - first;
      const int from = __shfl_sync(0xffffffffu, src, i < 0 || i >= n ? 0 : i);
      v[k] = make_uint4(0, 0, 0, 0);
      if (i >= 0 && i < n) v[k] = __ldg(reinterpret_cast<const uint4*>(x + (long long)from * p.stride));
    }
    uint8_t* const rec = p.cache[layer] + (((size_t)page * p.heads + head) * 2 + (is_v ? 1 : 0)) * kv4_record(D);
    uint16_t* const scales = reinterpret_cast<uint16_t*>(rec + kv4_codes(D));
    uint4 old[4];                          // V: what a page that stays in part holds
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      old[e] = make_uint4(0, 0, 0, 0);
      if (is_v && n < kPage && sub == 0) old[e] = reinterpret_cast<const uint4*>(rec + col * 64)[e];
    }
    uint32_t acc[2][8];                    // V: the words of this lane's dims
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[h][e] = 0u;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int token = k * kRowsAtOnce + sub;
      // (the same for the whole warp: nobody has a row of this step)
      if (k * kRowsAtOnce + kRowsAtOnce <= first || k * kRowsAtOnce >= first + n) continue;
      const bool mine = token >= first && token < first + n;
      // The largest of the block's values and of their negatives, as integers, where one of the two is above the other.
      const uint32_t flip = 0x80008000u;
      uint32_t up = __vmaxs2(__vmaxs2(v[k].x, v[k].y), __vmaxs2(v[k].z, v[k].w));
      uint32_t down = __vmaxs2(__vmaxs2(v[k].x ^ flip, v[k].y ^ flip), __vmaxs2(v[k].z ^ flip, v[k].w ^ flip));
      // low half: of the values, high half: of the negatives
      uint32_t most = __vmaxs2(__byte_perm(up, down, 0x5410), __byte_perm(up, down, 0x7632));
      most = __vmaxs2(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = __vmaxs2(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int hi = (int)(short)(most & 0xffffu), lo = (int)(short)(most >> 16);
      uint32_t key = hi > lo ? (uint32_t)hi << 6 : (uint32_t)lo << 6 | 1u;
      // ties of magnitude, what is no number, and magnitudes that the largest scale does not reach
      if (__any_sync(0xffffffffu, hi == lo || max(hi, lo) >= 0x7e80)) {
        key = top_key(v[k], (lane & 3) * 8);
        key = max(key, __shfl_xor_sync(0xffffffffu, key, 1));
        key = max(key, __shfl_xor_sync(0xffffffffu, key, 2));
        if (wild(v[k])) {
          any_wild = true;
          v[k] = make_uint4(tamed(v[k].x, key >> 6), tamed(v[k].y, key >> 6), tamed(v[k].z, key >> 6), tamed(v[k].w, key >> 6));
        }
        v[k] = make_uint4(reached(v[k].x), reached(v[k].y), reached(v[k].z), reached(v[k].w));
      }
      const uint32_t s = scale_of(key);
      const float inv = s == 0u ? 0.f : fast_rcp(bf16_value(s));
      if (mine && (lane & 3) == 0) {
        const int block = col >> 2;
        scales[is_v ? block * kPage + token : token * kBlocks + block] = (uint16_t)s;
      }
      const uint32_t c[4] = {codes2(v[k].x, inv), codes2(v[k].y, inv), codes2(v[k].z, inv), codes2(v[k].w, inv)};
      if (!is_v) {
        s_k[warp][(col >> 2) * (kPage * 4) + token * 4 + (col & 3)] = c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12;
      } else {
        // a dim's code into the half of its token's parity, four bits on for every two tokens
        const int h = k / (kSteps / 2);
        const bool odd = kRowsAtOnce == 1 ? (k & 1) : sub;
        const int shift = kRowsAtOnce == 1 ? 4 * ((k & 7) >> 1) : 4 * (k & 3);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[h][2 * e] |= __byte_perm(c[e], 0u, odd ? 0x1044 : 0x4410) << shift;
          acc[h][2 * e + 1] |= __byte_perm(c[e], 0u, odd ? 0x3244 : 0x4432) << shift;
        }
      }
    }
    if (any_wild) report(p.dev_status, SD_DEV_NOT_FINITE);
    if (!is_v) {
      __syncwarp();
      // 16-byte pieces: [block][token]
#pragma unroll
      for (int k = 0; k < kBlocks * kPage / 32; ++k) {
        const int e = k * 32 + lane, token = e % kPage;
        if (token >= first && token < first + n)
          reinterpret_cast<uint4*>(rec)[e] = reinterpret_cast<const uint4*>(s_k[warp])[e];
      }
      __syncwarp();
    } else {
      if (kRowsAtOnce == 2) {              // the other half of the lanes has the other tokens of the same dims
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[h][e] |= __shfl_xor_sync(0xffffffffu, acc[h][e], 16);
      }
      uint32_t keep[2] = {0u, 0u};         // codes of tokens that get no row
      if (n < kPage) {
#pragma unroll
        for (int t = 0; t < kPage; ++t)
          if (t < first || t >= first + n) keep[t >> 3] |= 15u << kv4_shift(t & 7);
      }
      uint4* at = reinterpret_cast<uint4*>(rec + col * 64);
      if (sub == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 o = make_uint4(acc[0][2 * e], acc[1][2 * e], acc[0][2 * e + 1], acc[1][2 * e + 1]);
          if (n < kPage)
            o = make_uint4((o.x & ~keep[0]) | (old[e].x & keep[0]), (o.y & ~keep[1]) | (old[e].y & keep[1]),
                           (o.z & ~keep[0]) | (old[e].z & keep[0]), (o.w & ~keep[1]) | (old[e].w & keep[1]));
          at[e] = o;
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads) kv4_read_kernel(const Kv4RowsParams p, const int window) {
  constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes, kBlocks = D / kKv4Block;
  const int layer = blockIdx.y, lane = threadIdx.x & 31;
  const int combo = blockIdx.z * kRowsWarps + (threadIdx.x >> 5);
  pdl_wait();
  if (combo >= 2 * p.heads) return;
  const int head = combo >> 1;
  const bool is_v = combo & 1;
  const int r0 = blockIdx.x * window, n = min(window, p.max_rows - r0);
  int mine = -1;
  if (lane < n) {
    mine = p.slots[r0 + lane];
    if (mine < -1 || mine / kPage >= p.num_pool_pages) {
      if (layer == 0 && combo == 0) report(p.dev_status, SD_DEV_BAD_SLOT);
      mine = -1;
    }
  }
  const int col = lane % kLanes, sub = lane / kLanes, block = col >> 2;
  __nv_bfloat16* out = (is_v ? p.v_rows[layer] : p.k_rows[layer]) + head * D + col * 8;
  const uint8_t* cache = p.cache[layer] + ((size_t)head * 2 + (is_v ? 1 : 0)) * kv4_record(D);
  const size_t page_bytes = (size_t)p.heads * 2 * kv4_record(D);
  bool bad = false;
  if (!is_v) {
    constexpr int kSteps = kPage / kRowsAtOnce;
    uint32_t w[kSteps], s[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = k * kRowsAtOnce + sub;
      const int slot = __shfl_sync(0xffffffffu, mine, i);
      w[k] = s[k] = 0u;
      if (slot >= 0) {
        const uint8_t* rec = cache + (size_t)(slot / kPage) * page_bytes;
        const int token = slot % kPage;
        w[k] = reinterpret_cast<const uint32_t*>(rec)[block * (kPage * 4) + token * 4 + (col & 3)];
        s[k] = reinterpret_cast<const uint16_t*>(rec + kv4_codes(D))[token * kBlocks + block];
      }
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = k * kRowsAtOnce + sub;
      const int slot = __shfl_sync(0xffffffffu, mine, i);
      const __nv_bfloat162 sc = kv4_scale2(kv4_sane(s[k] * 0x10001u, bad)), less = kv4_less(sc);
      if (slot >= 0)
        *reinterpret_cast<uint4*>(out + (long long)(r0 + i) * p.stride) =
            make_uint4(kv4_pair(w[k], 0, sc, less), kv4_pair(w[k], 1, sc, less), kv4_pair(w[k], 2, sc, less),
                       kv4_pair(w[k], 3, sc, less));
    }
  } else {
    // entry by entry; the lanes of a row hold the words of the page they are on
    uint4 w[4];
    int page = -1;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kRowsAtOnce) {
      const int i = i0 + sub;
      const int slot = __shfl_sync(0xffffffffu, mine, i & 31);
      if (i >= n || slot < 0) continue;
      const uint8_t* rec = cache + (size_t)(slot / kPage) * page_bytes;
      const int token = slot % kPage;
      if (slot / kPage != page) {
        page = slot / kPage;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = reinterpret_cast<const uint4*>(rec + col * 64)[e];
      }
      const uint32_t s = reinterpret_cast<const uint16_t*>(rec + kv4_codes(D))[block * kPage + token];
      const __nv_bfloat162 sc = kv4_scale2(kv4_sane(s * 0x10001u, bad)), less = kv4_less(sc);
      const int shift = kv4_shift(token & 7);
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = (token < 8 ? w[e].x : w[e].y) >> shift & 15u, b = (token < 8 ? w[e].z : w[e].w) >> shift & 15u;
        y[e] = kv4_pair(a | b << 16, 0, sc, less);
      }
      *reinterpret_cast<uint4*>(out + (long long)(r0 + i) * p.stride) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  if (bad) report(p.dev_status, SD_DEV_BAD_SCALE);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsParams& p, int dim, cudaStream_t st) {
  if (p.max_rows == 0) return cudaSuccess;
  // Rows per CTA: a row of its own while that fills the machine about twice over at most (single tokens of a batch, an
  // accepted path); for prompts sixteen, of which one begins a page.
  const int window = (long long)p.max_rows * p.num_layers <= 4 * kSMs ? 1 : kPage;
  // enough CTAs per window for one page's tasks, a warp each
  const int share = (2 * p.heads + kRowsWarps - 1) / kRowsWarps;
  const dim3 grid((p.max_rows + window - 1) / window, p.num_layers, share);
  if (dim == 256)
    kv4_append_kernel<256><<<grid, kRowsThreads, 0, st>>>(p, window);
  else
    kv4_append_kernel<128><<<grid, kRowsThreads, 0, st>>>(p, window);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsParams& p, int dim, cudaStream_t st) {
  if (p.max_rows == 0) return cudaSuccess;
  const int window = kPage;
  const int share = (2 * p.heads + kRowsWarps - 1) / kRowsWarps;
  const dim3 grid((p.max_rows + window - 1) / window, p.num_layers, share);
  return dim == 256 ? launch_pdl(kv4_read_kernel<256>, grid, dim3(kRowsThreads), 0, st, p, window)
                    : launch_pdl(kv4_read_kernel<128>, grid, dim3(kRowsThreads), 0, st, p, window);
}

}  // namespace sdv
