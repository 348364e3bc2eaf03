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
// One warp owns one (layer, K or V, half page, KV head): the half's new rows are
// in its registers, so bytes are read once, and V's words, which hold eight
// tokens each, are put together without a second writer.  A lane has eight
// consecutive dims: four lanes are a block, two shuffles its maximum.  K's words go through
// shared memory (a row's lie 256 bytes apart), so that its record leaves in
// 16-byte pieces; V's codes add up in halves of a word, two dims at a time.  Every warp finds its rows in the slot map for
// itself.  2 bytes read and 9/16 written a value, and some 18 instructions: 8191 rows of 4 heads of 256 dims take 16 us
// where their bytes take 6.4 (whole pages a warp, 128 registers: 17.6).  No bound is near: 54 % of the issue slots, 53 % of the
// ALU pipe and 21 % of HBM are in use; 80 registers leave an SM 24 warps, each of which loads its rows, then computes, then
// stores.  6 rows of 16 layers take 3.1, of which a launch is 2.
//
// Read.  One warp per (layer, K or V, KV head, eight entries of the slot map); V's
// words of a page are loaded once for the entries that lie on it.  16383 rows of 4 heads of 256 dims take 17 us, 0.75 of
// the copy rate; half of the instructions' rate is in use, so neither bound is near.  (V's scales of all entries first:
// 18.2.)
#include "kernels.h"
#include "kv4_format.cuh"

namespace sdv {
namespace {

constexpr int kRowsThreads = 128, kRowsWarps = kRowsThreads / 32;
constexpr int kReadRows = 8;             // entries of a warp of the read (of 16 layers x 8 sequences x 16 tokens: 16 4.4 us, 8 3.8, 4 4.2)

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
__global__ void __launch_bounds__(kRowsThreads, 6) kv4_append_kernel(const Kv4RowsParams p) {
  constexpr int kLanes = D / 8;            // lanes per row (8 values each)
  constexpr int kRowsAtOnce = 32 / kLanes; // rows a warp touches per step
  constexpr int kHalf = kPage / 2, kSteps = kHalf / kRowsAtOnce;
  constexpr int kBlocks = D / kKv4Block;
  __shared__ __align__(16) uint32_t s_k[kRowsWarps][kHalf * D / 8];
  const int layer = blockIdx.y, r_base = blockIdx.x * kPage;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int combo = blockIdx.z * kRowsWarps + warp;
  if (combo >= 4 * p.heads) return;
  const int head = combo >> 2, half = combo & 1;      // tokens 0..7 of the page, or 8..15
  const bool is_v = combo & 2;
  const int col = lane % kLanes, sub = lane / kLanes;
  pdl_wait();
  // Sixteen entries, and the 16 behind them, one a lane: every warp finds its groups for itself, in one latency.
  int slot = -1, src = -1, prev = -1;
  if (lane < p.max_rows - r_base) {
    slot = p.slots[r_base + lane];
    src = p.rows != nullptr ? p.rows[r_base + lane] : r_base + lane;
  }
  if (lane == 0 && r_base > 0) prev = p.slots[r_base - 1];
  const int up = __shfl_up_sync(0xffffffffu, slot, 1);
  if (lane > 0) prev = up;
  bool lead = false;
  if (lane < kPage) {
    if (slot < -1 || slot / kPage >= p.num_pool_pages) {
      if (layer == 0 && combo == 0) report(p.dev_status, SD_DEV_BAD_SLOT);
    } else if (slot >= 0) {
      lead = prev < 0 || prev / kPage != slot / kPage;
    }
  }
#pragma unroll 1
  for (uint32_t leads = __ballot_sync(0xffffffffu, lead); leads != 0u; leads &= leads - 1u) {
    // the group: the following rows on the same page, which must rise by one (a seventeenth cannot)
    const int l0 = __ffs(leads) - 1;
    const int slot0 = __shfl_sync(0xffffffffu, slot, l0), page = slot0 / kPage, first = slot0 % kPage;
    const bool same = lane >= l0 && slot >= 0 && slot / kPage == page;
    const int n = __ffs(~(__ballot_sync(0xffffffffu, same) >> l0 & 0x1ffffu)) - 1;   // 1..17
    const int i_lane = lane - l0;
    const bool wrong = i_lane >= 0 && i_lane < n && (slot != slot0 + i_lane || src < 0 || src >= p.num_src_rows);
    if (__any_sync(0xffffffffu, wrong)) {
      if (lane == 0 && layer == 0) report(p.dev_status, SD_DEV_BAD_SLOT);
      continue;
    }
    // the half's tokens that get a row
    const int lo = max(first, half * kHalf) - half * kHalf, hi = min(first + n, half * kHalf + kHalf) - half * kHalf;
    if (lo >= hi) continue;
    const __nv_bfloat16* x = (is_v ? p.v_rows[layer] : p.k_rows[layer]) + head * D + col * 8;
    // A lane's rows by their token in the half: step k is token k * kRowsAtOnce + sub.
    uint4 v[kSteps];
    bool any_wild = false;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int token = k * kRowsAtOnce + sub;
      const bool mine = token >= lo && token < hi;
      const int from = __shfl_sync(0xffffffffu, src, mine ? l0 + token + half * kHalf - first : l0);
      v[k] = make_uint4(0, 0, 0, 0);
      if (mine) v[k] = __ldg(reinterpret_cast<const uint4*>(x + (long long)from * p.stride));
    }
    uint8_t* const rec = p.cache[layer] + (((size_t)page * p.heads + head) * 2 + (is_v ? 1 : 0)) * kv4_record(D);
    uint16_t* const scales = reinterpret_cast<uint16_t*>(rec + kv4_codes(D));
    const bool whole = lo == 0 && hi == kHalf;
    uint32_t* const words = reinterpret_cast<uint32_t*>(rec) + col * 16 + half;      // V: this lane's dims, two words apart
    // V: codes of two dims in the halves of a sum, four bits on for every second token; sums of the even and the odd tokens
    // (over 128 dims the two halves of the warp have one each)
    constexpr int kSums = 2 / kRowsAtOnce;
    uint32_t acc[kSums][4], old[8];        // old: what a half page that stays in part holds
#pragma unroll
    for (int e = 0; e < 4 * kSums; ++e) acc[e / 4][e % 4] = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      old[e] = 0u;
      if (is_v && !whole && sub == 0) old[e] = words[2 * e];
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int token = k * kRowsAtOnce + sub;
      // (the same for the whole warp: nobody has a row of this step)
      if (k * kRowsAtOnce + kRowsAtOnce <= lo || k * kRowsAtOnce >= hi) continue;
      const bool mine = token >= lo && token < hi;
      // The largest of the block's values and of their negatives, as integers, where one of the two is above the other.
      const uint32_t flip = 0x80008000u;
      uint32_t up = __vmaxs2(__vmaxs2(v[k].x, v[k].y), __vmaxs2(v[k].z, v[k].w));
      uint32_t down = __vmaxs2(__vmaxs2(v[k].x ^ flip, v[k].y ^ flip), __vmaxs2(v[k].z ^ flip, v[k].w ^ flip));
      // low half: of the values, high half: of the negatives
      uint32_t most = __vmaxs2(__byte_perm(up, down, 0x5410), __byte_perm(up, down, 0x7632));
      most = __vmaxs2(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = __vmaxs2(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int pos = (int)(short)(most & 0xffffu), neg = (int)(short)(most >> 16);
      uint32_t key = pos > neg ? (uint32_t)pos << 6 : (uint32_t)neg << 6 | 1u;
      // ties of magnitude, what is no number, and magnitudes that the largest scale does not reach
      if (__any_sync(0xffffffffu, pos == neg || max(pos, neg) >= 0x7e80)) {
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
        const int block = col >> 2, in_page = token + half * kHalf;
        scales[is_v ? block * kPage + in_page : in_page * kBlocks + block] = (uint16_t)s;
      }
      const uint32_t c[4] = {codes2(v[k].x, inv), codes2(v[k].y, inv), codes2(v[k].z, inv), codes2(v[k].w, inv)};
      if (!is_v) {
        s_k[warp][(col >> 2) * (kHalf * 4) + token * 4 + (col & 3)] = c[0] + (c[1] << 4) + (c[2] << 8) + (c[3] << 12);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k % kSums][e] += c[e] << (4 * (k / kSums));
      }
    }
    if (any_wild) report(p.dev_status, SD_DEV_NOT_FINITE);
    if (!is_v) {
      __syncwarp();
      // 16-byte pieces: [block][token]
#pragma unroll
      for (int k = 0; k < kBlocks * kHalf / 32; ++k) {
        const int e = k * 32 + lane, token = e % kHalf;
        if (token >= lo && token < hi)
          reinterpret_cast<uint4*>(rec)[e / kHalf * kPage + half * kHalf + token] = reinterpret_cast<const uint4*>(s_k[warp])[e];
      }
      __syncwarp();
    } else {
      uint32_t word[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t even = acc[0][e], odd = kSums == 2 ? acc[kSums - 1][e] : __shfl_xor_sync(0xffffffffu, even, 16);
        word[2 * e] = __byte_perm(even, odd, 0x5410);
        word[2 * e + 1] = __byte_perm(even, odd, 0x7632);
      }
      uint32_t keep = 0u;                  // codes of tokens that get no row
      if (!whole) {
#pragma unroll
        for (int t = 0; t < kHalf; ++t)
          if (t < lo || t >= hi) keep |= 15u << kv4_shift(t);
      }
      if (sub == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) words[2 * e] = (word[e] & ~keep) | (old[e] & keep);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads) kv4_read_kernel(const Kv4RowsParams p) {
  constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes, kBlocks = D / kKv4Block;
  const int layer = blockIdx.y, lane = threadIdx.x & 31;
  const int combo = blockIdx.z * kRowsWarps + (threadIdx.x >> 5);
  pdl_wait();
  if (combo >= 2 * p.heads) return;
  const int head = combo >> 1;
  const bool is_v = combo & 1;
  const int r0 = blockIdx.x * kReadRows, n = min(kReadRows, p.max_rows - r0);
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
    constexpr int kSteps = kReadRows / kRowsAtOnce;
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
  // a warp for each half page, K or V and head of sixteen entries, of which one or two begin a page
  const int share = (4 * p.heads + kRowsWarps - 1) / kRowsWarps;
  const dim3 grid((p.max_rows - 1) / kPage + 1, p.num_layers, share);
  return dim == 256 ? launch_pdl(kv4_append_kernel<256>, grid, dim3(kRowsThreads), 0, st, p)
                    : launch_pdl(kv4_append_kernel<128>, grid, dim3(kRowsThreads), 0, st, p);
}

cudaError_t launch_kv4_read(const Kv4RowsParams& p, int dim, cudaStream_t st) {
  if (p.max_rows == 0) return cudaSuccess;
  const int share = (2 * p.heads + kRowsWarps - 1) / kRowsWarps;
  const dim3 grid((p.max_rows - 1) / kReadRows + 1, p.num_layers, share);
  return dim == 256 ? launch_pdl(kv4_read_kernel<256>, grid, dim3(kRowsThreads), 0, st, p)
                    : launch_pdl(kv4_read_kernel<128>, grid, dim3(kRowsThreads), 0, st, p);
}

}  // namespace sdv
