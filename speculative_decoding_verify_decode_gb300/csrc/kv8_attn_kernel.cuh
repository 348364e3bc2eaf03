// Verify attention over the 8-bit block-scaled cache (include/sd_kv8.h:
// sd_kv8_attn): tcgen05 products straight on the cache's e4m3 codes.
//
// The mathematics.  A query column q is one (draft node, query head) pair of a
// KV head; a key is a context token t with codes k_t, v_t and block scales
// a_t (K) and c_t (V), or a draft node.  With s = cap(scale q.k) + bias in
// base 2 and a running reference m of the column,
//   e = 2^(s - m),   l += e,   O += (e c_t) v_t,   out = O / l,
// so a V scale goes into the weight and a K scale into the score, each one
// multiplication per score, constant along a token row, and the tensor core
// never sees anything but codes.  m is the running maximum of s + log2 c_t
// less kHead: the weights e c_t stay at or below 2^kHead however uneven the
// blocks are, and m moves (with O and l rescaled) only when a weight passes
// kTop, the largest e4m3 value.
//
// The 8-bit operands.  K and V are exact as they lie.  A bf16 query is two
// e4m3 terms (a power-of-two scale per row, then the rounded value and the
// rounded rest: 8 significant bits, off by at most 2^-18 of the row's amax);
// both multiply the same K tile into the same accumulator.  A weight is an
// e4m3 term and an e5m2 rest (2^-4 times 2^-3: at most 2^-7 off, about 2^-9.5
// in the mean square; e5m2 so that the rest of small weights keeps its
// exponent range, down to 2^-16).  l sums the unrounded fp32 weights.  Draft
// keys and values are bf16 and take two e4m3 terms each, four products.
//
// What bounds it.  Bytes: 2 D per token and KV head (codes of K and V), read
// once per CTA column part.  Widening the codes to f16 in shared memory, the
// alternative, moves about 500 KB of shared memory per 128-token tile; here a
// tile's codes are written by TMA and read by the tensor core only.
//
// Work split.  The 128-token tiles of every (sequence, KV head, head part)
// segment, its draft block in front as one more tile, form one line of units
// that is cut into equal pieces, one per CTA, on the device from ctx_lens: no
// host knowledge of the lengths, no idle CTA on a ragged batch.  A segment cut
// by piece borders leaves bf16 partial outputs and fp32 log-sum-exps for the
// merge; one that lies in a single piece is written directly.
//
// Per tile (tokens are the MMA's M; NQ columns):
//   S[128 tok][NQ]     = K_tile . (Qhi + Qlo)^T      K-major, K = 32 a step
//   O^T[D][NQ]        += V_tile^T . (Phi + Plo)^T    M = 128 dims a product, MN-major
// Warps: 0-7 softmax (lane quarter = warp % 4, column half = warp / 4; thread =
// token row), which also stage Q and the draft block and write the results; 8
// loads K and the block scales, 9 loads V, 10 issues QK, 11 issues PV.
// Every wait is bounded; on expiry the kernel reports SD_DEV_TIMEOUT and ends.
#pragma once

#include <cstddef>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace sdv {
namespace {

constexpr int kKvThreads = 384;
constexpr int kWarpK = 8, kWarpV = 9, kWarpQK = 10, kWarpPV = 11;
constexpr int kTile = kTileTokens;
constexpr float kHead = 6.0f;          // the largest weight sits at 2^6 when m is exact
constexpr float kTop = 448.0f;         // weights beyond it move m
constexpr float kNone = -1.0e30f;      // m before any visible key
constexpr float kScaleLo = 0x1p-100f, kScaleHi = 0x1p100f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSmemBytes = 232448;     // 227 KB of dynamic shared memory per CTA
constexpr int kScaleStages = 6;

// TIGHT: 144 columns of 256 dims leave 7 KB beside the operands and seven 16 KB half tiles.
template <int NQ, bool MOD, bool TIGHT>
struct KvSmall {
  static constexpr int kBars = TIGHT ? 24 : 40;
  float f[NQ];             // score factor of a column: its query scale times the softmax scale, base 2
  float m[NQ];             // the column's reference m
  float alpha[NQ];         // rescale factor of the current tile; 1 / l in the epilogue
  float slope[MOD ? NQ : 4];   // distance bias (base 2) and depth of the column's node
  float dep[MOD ? NQ : 4];
  float red[4][NQ];        // per lane quarter: column maxima of a tile; column sums in the epilogue
  float scale[kScaleStages][16];   // K scales, then V scales, of a tile's eight pages
  float row_k[kMaxNodes], row_v[kMaxNodes];   // scales of the draft block's rows
  unsigned long long anc[kMaxNodes];          // bit r: node r is on the node's root path
  uint64_t bar[kBars];
  int cum[kMaxBatch + 1];  // first unit of each sequence
  int scan[8];
  int8_t par[kMaxNodes];
  int8_t depth[kMaxNodes];
  int flag[2][2][4];       // [column half][tile parity][lane quarter]: a weight passed kTop
  uint32_t tmem;
  int abort;
};

template <int D, int HC, bool MOD>
struct Kv {
  using Small = KvSmall<HC == 5 ? 144 : 32 * HC, MOD, HC == 5 && D == 256>;
  static constexpr int NQ = HC == 5 ? 144 : 32 * HC;      // query columns
  static constexpr int MH = D / 128;                      // 128-dim blocks
  static constexpr int NS = (2 + MH) * NQ <= 512 ? 2 : 1; // S buffers in tensor memory
  static constexpr int kCols = (NS + MH) * NQ;
  static constexpr int kTmem = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr int kGroupBytes = MH * 1024;           // 8 token rows
  static constexpr int kPageBytes = 2 * kGroupBytes;      // a page of one KV head
  static constexpr int kHalf = 4 * kPageBytes;            // 64 tokens
  static constexpr int kTileBytes = 2 * kHalf;
  static constexpr int kQTerm = NQ * D, kQBytes = 2 * kQTerm;
  static constexpr int kPTerm = NQ * kTile, kPBytes = 2 * kPTerm;
  static constexpr int kLeft = (kSmemBytes - kQBytes - kPBytes - (int)sizeof(Small)) / kHalf;
  static constexpr int kUnits = kLeft > 16 ? 16 : kLeft;  // half tiles of ring
  static constexpr int KS = kUnits / 4 < 2 ? 2 : kUnits / 4;   // K tiles
  static constexpr int VS = kUnits - 2 * KS;                   // V half tiles
  static constexpr size_t kSmem = (size_t)kQBytes + kPBytes + KS * kTileBytes + VS * kHalf + sizeof(Small);
  static_assert(VS >= 3, "the V ring holds more than a tile");
  static_assert(KS + NS <= kScaleStages, "scale stages");
  static_assert(kSmem <= (size_t)kSmemBytes, "shared memory over 227 KB");
};

// ------------------------------------------------------------ small pieces

__device__ __forceinline__ uint64_t noswz_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}
// kind::f8f6f4, fp32 accumulators: A e4m3, B e4m3 or e5m2.
__device__ __forceinline__ uint32_t f8_idesc(int n, int a_mn, int b_mn, bool b_e5m2) {
  return (1u << 4) | (b_e5m2 ? 1u << 10 : 0u) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void umma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tma_page8(uint32_t dst, const CUtensorMap* map, int w, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3}], [%4], %5;"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(w), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint32_t r;
  asm("{ .reg .b16 t; cvt.rn.satfinite.e4m3x2.f32 t, %1, %2; cvt.u32.u16 %0, t; }" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_val(uint32_t codes) {
  uint32_t h;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
// Four weights (two pairs, columns in order) as four e4m3 codes and four e5m2 codes of the rest.
__device__ __forceinline__ void split4(float2 w0, float2 w1, uint32_t& hi, uint32_t& lo) {
  asm("{ .reg .b32 a, b, c, d; .reg .b16 s, t, u, v;\n\t"
      "cvt.rn.f16x2.f32 a, %3, %2;\n\t"
      "cvt.rn.f16x2.f32 b, %5, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 s, a;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 t, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 c, s;\n\t"
      "cvt.rn.f16x2.e4m3x2 d, t;\n\t"
      "sub.rn.f16x2 c, a, c;\n\t"
      "sub.rn.f16x2 d, b, d;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 u, c;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 v, d;\n\t"
      "mov.b32 %0, {s, t};\n\t"
      "mov.b32 %1, {u, v}; }"
      : "=r"(hi), "=r"(lo)
      : "f"(w0.x), "f"(w0.y), "f"(w1.x), "f"(w1.y));
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Reduce 16 values per lane over the warp: lane L ends with the result for value L % 16.
template <bool MAX>
__device__ __forceinline__ float reduce16(float (&v)[16], int lane) {
#pragma unroll
  for (int half = 8; half >= 1; half >>= 1) {
    const bool up = (lane & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, half);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
  return MAX ? fmaxf(v[0], got) : v[0] + got;
}

// Eight bf16 as two e4m3 terms (hi + lo) of x * 2^-e.
__device__ __forceinline__ void split8(const uint4 x, float inv, uint2& hi, uint2& lo) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    v.x *= inv;
    v.y *= inv;
    h[i] = e4m3x2_of(v.x, v.y);
    const float2 b = e4m3x2_val(h[i]);
    l[i] = e4m3x2_of(v.x - b.x, v.y - b.y);
  }
  hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}
// Largest bf16 magnitude of a chunk, as bits (infinities and NaN sort above the finite values).
__device__ __forceinline__ uint32_t amax_bits(const uint4 x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}
// Exponent e of the smallest 2^e with amax <= 448 * 2^e (clamped to the block scales' range).
__device__ __forceinline__ int exp_of(uint32_t bits) {
  return min(100, max(-100, (int)(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0)));
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// One CTA's share of one segment.
struct Piece {
  int b, g, c;         // sequence, KV head, head part
  int seg;
  int L, base;         // context length; first position the tiles cover
  int first, tiles;    // first tile of the segment (0: the draft block) and how many
  bool whole;          // the segment lies in this piece alone
};

template <int D, int HC, bool MOD>
__global__ void __launch_bounds__(kKvThreads, 1)
kv8_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const Kv8AttnParams p, const BatchDesc bd) {
  using K = Kv<D, HC, MOD>;
  constexpr int NQ = K::NQ, MH = K::MH, NS = K::NS, KS = K::KS, VS = K::VS;
  using Sm = typename K::Small;
  constexpr int B_KF = 0, B_KE = KS, B_VF = 2 * KS, B_VE = B_VF + VS, B_SC = B_VE + VS, B_SF = B_SC + KS + NS,
                B_SE = B_SF + NS, B_PF = B_SE + NS, B_OD = B_PF + 1, B_Q = B_PF + 2, B_G0 = B_PF + 3, B_G1 = B_PF + 4,
                B_ALL = B_PF + 5;
  constexpr int kNumBars = B_ALL + 1;
  static_assert(kNumBars <= Sm::kBars, "barriers");
  constexpr int SC = KS + NS;   // scale stages: see the K producer
  extern __shared__ __align__(1024) uint8_t smem8[];
  uint8_t* sQ = smem8;
  uint8_t* sK = sQ + K::kQBytes;
  uint8_t* sV = sK + KS * K::kTileBytes;
  uint8_t* sP = sV + VS * K::kHalf;
  Sm* sm = reinterpret_cast<Sm*>(sP + K::kPBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem8) & 1023u) {   // not expected; refuse rather than mis-swizzle
    if (tid == 0) report(p.dev_status, SD_DEV_TIMEOUT);
    return;
  }

  // ---------------------------------------------------------------- the line of units
  const int parts = p.hkv * p.hparts;   // segments per sequence
  auto ctx_of = [&](int b) {
    const int L = p.ctx_lens[b];
    return L < 0 ? 0 : min(L, p.max_pages * kPage);
  };
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(smem_u32(&sm->bar[i]), i == B_PF || i == B_ALL || (i >= B_SE && i < B_SE + NS) ? 8u
                                       : i == B_G0 || i == B_G1 ? 4u : 1u);
    sm->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  {
    int n = 0;
    if (tid < bd.batch) {
      const int raw = p.ctx_lens[tid], L = ctx_of(tid);
      if (blockIdx.x == 0 && raw != L) report(p.dev_status, SD_DEV_BAD_CTX);
      n = (1 + (L - window_base(L, p.window, kTile) + kTile - 1) / kTile) * parts;
    }
    int incl = n;
    if (warp < 8) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += up;
      }
      if (lane == 31) sm->scan[warp] = incl;
    }
    __syncthreads();
    if (warp < 8) {
      for (int w = 0; w < warp; ++w) incl += sm->scan[w];
      if (tid == 0) sm->cum[0] = 0;
      if (tid < bd.batch) sm->cum[tid + 1] = incl;
    }
  }
  if (warp == kWarpQK) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem)),
                 "n"(K::kTmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int total = sm->cum[bd.batch];
  const int per = (total + gridDim.x - 1) / gridDim.x;
  const int u_begin = min(total, (int)blockIdx.x * per), u_end = min(total, u_begin + per);
  if (blockIdx.x == 0) {   // for the merge
    for (int i = tid; i <= bd.batch; i += kKvThreads) p.cum[i] = sm->cum[i];
  }
  // The piece that begins at unit u.
  auto piece_at = [&](int u) {
    Piece pc;
    int lo = 0, hi = bd.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sm->cum[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const int units = (sm->cum[lo + 1] - sm->cum[lo]) / parts;
    const int rem = u - sm->cum[lo], s = rem / units;
    pc.b = lo;
    pc.g = s / p.hparts;
    pc.c = s - pc.g * p.hparts;
    pc.seg = lo * parts + s;
    pc.first = rem - s * units;
    pc.tiles = min(units - pc.first, u_end - u);
    pc.whole = pc.tiles == units;
    pc.L = ctx_of(lo);
    pc.base = window_base(pc.L, p.window, kTile);
    return pc;
  };
  const uint32_t bars = smem_u32(&sm->bar[0]);
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto wait = [&](int i, int n) { return mbar_wait(bar(i), (uint32_t)n & 1u, &sm->abort, p.dev_status); };
  // for whole warps: one answer, so that a warp leaves as one
  auto spin = [&](int i, int n) {
    return __all_sync(0xffffffffu, mbar_spin(bar(i), (uint32_t)n & 1u, &sm->abort, p.dev_status)) != 0;
  };
  const uint32_t tmem = sm->tmem;
  const uint32_t kColO = NS * NQ;   // O^T behind the S buffers

  if (warp == kWarpK || warp == kWarpV) {
    // ------------------------------------------------------------ producers
    const bool is_k = warp == kWarpK;
    const CUtensorMap* map = is_k ? &tm_k : &tm_v;
    const uint64_t policy = l2_evict_first();
    int it = 0;         // tiles so far (the draft block's among them: staged by the softmax warps)
    bool ok = true;
    for (int u = u_begin; u < u_end && ok;) {
      const Piece pc = piece_at(u);
      u += pc.tiles;
      const int* row = p.page_table + (size_t)pc.b * p.max_pages;
      // page id of lane l's page of the tile that begins at t0 (-1: behind the context)
      auto fetch = [&](int t0) {
        const int pos = t0 + (lane & 7) * kPage;
        return pos < pc.L && (lane < 8 || is_k) && lane < 16 ? row[pos / kPage] : -1;
      };
      auto t0_of = [&](int i) { return pc.base + (pc.first + i - 1) * kTile; };
      const int i0 = pc.first == 0 ? 1 : 0;
      if (i0) {
        // the draft tile is staged by the softmax warps: its scale stage passes by empty, in its turn
        if (is_k) {
          ok = __all_sync(0xffffffffu, wait(B_KE + it % KS, it / KS + 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive(bar(B_SC + it % SC));
        }
        ++it;
      }
      int page_next = i0 < pc.tiles ? fetch(t0_of(i0)) : -1;
      for (int i = i0; i < pc.tiles && ok; ++i, ++it) {
        const int t0 = t0_of(i);
        const int valid = min(kTile, pc.L - t0);
        int page = page_next;
        page_next = i + 1 < pc.tiles ? fetch(t0_of(i + 1)) : -1;
        const bool in_ctx = lane < 16 && (lane & 7) * kPage < valid;
        const bool bad = in_ctx && (page < 0 || page >= p.num_pool_pages);
        if (bad) {
          if (is_k && lane < 8) report(p.dev_status, SD_DEV_BAD_PAGE);
          page = -1;
        }
        if (is_k) {
          // Block scales: lanes 0-7 those of K, 8-15 those of V.  A stage may be rewritten once the
          // softmax has read the scores of the tile KS + NS before, which the wait on K_EMPTY implies
          // (that tile's successor by NS has been multiplied).
          float sc = 1.f;
          if (in_ctx && page >= 0) {
            sc = __ldg((lane < 8 ? p.k_scales : p.v_scales) + (size_t)page * p.hkv + pc.g);
            if (!(sc >= kScaleLo && sc <= kScaleHi)) {
              report(p.dev_status, SD_DEV_BAD_SCALE);
              sc = sc > kScaleHi ? kScaleHi : kScaleLo;
            }
          }
          const int slot = it % KS;
          ok = wait(B_KE + slot, it / KS + 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* dst = sK + slot * K::kTileBytes;
          const uint32_t zero = __ballot_sync(0xffffffffu, lane < 8 && bad);
          if (zero != 0u) {
            for (uint32_t z = zero; z != 0u; z &= z - 1u)
              for (int e = lane; e < K::kPageBytes / 16; e += 32)
                reinterpret_cast<uint4*>(dst + (__ffs(z) - 1) * K::kPageBytes)[e] = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
          }
          const bool load = lane < 8 && page >= 0;
          const uint32_t mask = __ballot_sync(0xffffffffu, load);
          if (lane == 0) mbar_expect_tx(bar(B_KF + slot), (uint32_t)__popc(mask) * (uint32_t)K::kPageBytes);
          __syncwarp();
          if (load) tma_page8(smem_u32(dst + lane * K::kPageBytes), map, (page * p.hkv + pc.g) * 2, bar(B_KF + slot), policy);
          if (lane < 16) sm->scale[it % SC][lane] = sc;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_SC + it % SC));
        } else {
          // V: two halves of 64 tokens.  Rows that nobody sees must be zeros, not whatever lies there (a weight
          // of 0 times a NaN code is NaN): pages with such rows, and those that only some nodes of a tree see
          // through a window, go through plain loads, the rest by TMA.
          const int lo = p.window > 0 ? pc.L - p.window + 1 : 0;          // the root's oldest visible position
          for (int h = 0; h < 2; ++h) {
            const int fill = 2 * it + h, slot = fill % VS;
            ok = wait(B_VE + slot, fill / VS + 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint8_t* dst = sV + slot * K::kHalf;
            const int rows = min(64, valid - h * 64);
            const int steps = rows > 0 ? (rows + 31) / 32 * 2 : 0;        // pages up to the last 32-token step
            const int j = lane - 4 * h;
            const bool mine = lane >= 4 * h && j < steps && lane < 4 * h + 4;
            const int pos = t0 + lane * kPage;
            const bool plain = mine && (page < 0 || pos + kPage > pc.L || pos < lo + (p.window > 0 ? kMaxNodes : 0));
            const uint32_t slow = __ballot_sync(0xffffffffu, plain);
            for (uint32_t z = slow; z != 0u; z &= z - 1u) {
              const int l = __ffs(z) - 1;
              const int pg = __shfl_sync(0xffffffffu, page, l);
              for (int e = lane; e < kPage * D / 16; e += 32) {
                const int r = e / (D / 16), ch = e % (D / 16), t = t0 + l * kPage + r;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (pg >= 0 && t >= lo && t < pc.L) {
                  v = __ldg(reinterpret_cast<const uint4*>(p.v_cache + (((size_t)pg * p.hkv + pc.g) * kPage + r) * D) + ch);
                  if (p.window > 0 && t < lo + kMaxNodes) {   // NaN codes: the softmax makes the row's scores NaN instead
                    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) w[i4] &= ~__vcmpeq4(w[i4] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                  }
                }
                *reinterpret_cast<uint4*>(dst + ((l - 4 * h) * 2 + (r >> 3)) * K::kGroupBytes + (ch >> 3) * 1024 +
                                          (r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
              }
            }
            if (slow != 0u) fence_async_smem();
            __syncwarp();
            const bool load = mine && !plain;
            const uint32_t mask = __ballot_sync(0xffffffffu, load);
            if (lane == 0) mbar_expect_tx(bar(B_VF + slot), (uint32_t)__popc(mask) * (uint32_t)K::kPageBytes);
            __syncwarp();
            if (load) tma_page8(smem_u32(dst + j * K::kPageBytes), map, (page * p.hkv + pc.g) * 2, bar(B_VF + slot), policy);
            __syncwarp();
          }
        }
      }
    }
    // After an abort no copy may still be landing when the CTA ends: wait, bounded, for the last fills.
    if (lane == 0 && *(volatile int*)&sm->abort) {
      const int slots = is_k ? KS : VS, fills = is_k ? it : 2 * it;
      for (int s = 0; s < slots; ++s) {
        for (int back = 0; back < 2; ++back) {   // the last fill of the slot, and the one that may be under way
          const int n = (fills + 1 - s) / slots - back;
          if (n < 0) continue;
          const long long t0 = clock64();
          while (!mbar_test(bar((is_k ? B_KF : B_VF) + s), (uint32_t)n & 1u) && clock64() - t0 < kWaitCycles / 64) {
          }
        }
      }
    }
  } else if (warp == kWarpQK) {
    // ------------------------------------------------------------ QK issuer
    if (lane == 0) {
      int it = 0, np = 0;
      bool ok = true;
      for (int u = u_begin; u < u_end && ok; ++np) {
        const Piece pc = piece_at(u);
        u += pc.tiles;
        const int n_nodes = bd.q_indptr[pc.b + 1] - bd.q_indptr[pc.b];
        const int nq = (min(p.hpc, p.group - pc.c * p.hpc) * n_nodes + 15) & ~15;
        const uint32_t idesc = f8_idesc(nq, 0, 0, false);
        ok = wait(B_Q, np);
        for (int i = 0; i < pc.tiles && ok; ++i, ++it) {
          ok = wait(B_SE + it % NS, it / NS + 1) && wait(B_KF + it % KS, it / KS);
          if (!ok) break;
          tc_fence_after();
          const uint32_t k0 = smem_u32(sK + it % KS * K::kTileBytes), q0 = smem_u32(sQ);
          const uint32_t d = tmem + (it % NS) * NQ;
          // the draft block: rows 0-63 the keys' first terms, rows 64-127 the second (both onto rows 0-63 of S; the
          // other rows of S then hold nothing and are masked)
          const int terms = pc.first + i == 0 ? 2 : 1;
          for (int kt = 0; kt < terms; ++kt) {
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              const uint32_t off = (kk & 3) * 32;
              const uint64_t a = sw128_desc(k0 + kt * 8 * K::kGroupBytes + (kk >> 2) * 1024 + off, 16, K::kGroupBytes);
#pragma unroll
              for (int t = 0; t < 2; ++t)
                umma8(d, a, sw128_desc(q0 + t * K::kQTerm + (kk >> 2) * NQ * 128 + off, 16, 1024), idesc,
                      kt + kk + t > 0 ? 1u : 0u);
            }
          }
          umma_commit(bar(B_KE + it % KS));
          umma_commit(bar(B_SF + it % NS));
        }
      }
    }
  } else if (warp == kWarpPV) {
    // ------------------------------------------------------------ PV issuer
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int u = u_begin; u < u_end && ok;) {
        const Piece pc = piece_at(u);
        u += pc.tiles;
        const int n_nodes = bd.q_indptr[pc.b + 1] - bd.q_indptr[pc.b];
        const int nq = (min(p.hpc, p.group - pc.c * p.hpc) * n_nodes + 15) & ~15;
        const uint32_t id_hi = f8_idesc(nq, 1, 1, false), id_lo = f8_idesc(nq, 1, 1, true);
        for (int i = 0; i < pc.tiles && ok; ++i, ++it) {
          const bool draft = pc.first + i == 0;
          const int valid = draft ? n_nodes : min(kTile, pc.L - (pc.base + (pc.first + i - 1) * kTile));
          ok = wait(B_PF, it);
          for (int h = 0; h < 2 && ok; ++h) {
            const int fill = 2 * it + h, slot = fill % VS;
            ok = wait(B_VF + slot, fill / VS);
            if (!ok) break;
            tc_fence_after();
            // the draft block: half 0 the values' first terms, half 1 the second, both weighed by rows 0-63 of P
            const int rows = draft ? valid : min(64, valid - h * 64);
            const uint32_t v0 = smem_u32(sV + slot * K::kHalf);
            const uint32_t p0 = smem_u32(sP) + (draft ? 0 : h * 64 * 16);
            for (int ks = 0; ks * 32 < rows; ++ks) {
              const uint32_t first = i > 0 || h > 0 || ks > 0 ? 1u : 0u;
#pragma unroll
              for (int mb = 0; mb < MH; ++mb) {
                const uint64_t a = sw128_desc(v0 + ks * 4 * K::kGroupBytes + mb * 1024, 1024, K::kGroupBytes);
                // P: 16-column chunks of 128 token rows x 16 bytes; MN-major without a swizzle
                const uint32_t d = tmem + kColO + mb * NQ;
                umma8(d, a, noswz_desc(p0 + ks * 512, 128, kTile * 16), id_hi, first);
                umma8(d, a, noswz_desc(p0 + K::kPTerm + ks * 512, 128, kTile * 16), id_lo, 1u);
              }
            }
            umma_commit(bar(B_VE + slot));
          }
          if (ok) umma_commit(bar(B_OD));
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warps
    const int half = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;                       // token row of S; dim (mod 128) of O^T
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    int n_all = 0, n_grp = 0;
    auto sync_all = [&]() -> bool {      // the eight softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_ALL));
      return spin(B_ALL, n_all++);
    };
    auto sync_half = [&]() -> bool {     // the four warps of this column half
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_G0 + half));
      return spin(B_G0 + half, n_grp++);
    };
    int it = 0;
    bool ok = true;
    for (int u = u_begin; u < u_end && ok;) {
      const Piece pc = piece_at(u);
      u += pc.tiles;
      const int q0 = bd.q_indptr[pc.b], n_nodes = bd.q_indptr[pc.b + 1] - q0;
      const int hpc = min(p.hpc, p.group - pc.c * p.hpc);
      const int head0 = pc.g * p.group + pc.c * p.hpc;
      const int rows = hpc * n_nodes, nc = (rows + 15) / 16;
      const int c_first = half ? (nc + 1) / 2 : 0, mine = half ? nc / 2 : (nc + 1) / 2;   // 16-column chunks
      const int col0 = c_first * 16;
      const bool has_draft = pc.first == 0;
      // ---------------------------------------------------------- staging: Q, the tree, the draft block
      // (the previous piece's products have all finished: its last O_DONE was waited for)
      if (tid < n_nodes) {
        const int up = p.parents[q0 + tid];
        sm->par[tid] = (int8_t)(up < -1 || up >= kMaxNodes ? -2 : up);
      }
      {
        constexpr int LPR = D / 8, RPW = 32 / LPR;      // lanes per row, rows per warp and load
        constexpr int U = 6;
        const int sub = lane / LPR, ch = lane % LPR;    // 8-value chunk of the row
        const int n_draft = has_draft ? n_nodes : 0;
        const int n_q = nc * 16, n_stage = n_q + 2 * n_draft;
        if (has_draft) {
          // the ring slots of the draft tile, once their previous contents have been multiplied
          ok = spin(B_KE + it % KS, it / KS + 1) && spin(B_VE + 2 * it % VS, 2 * it / VS + 1) &&
               spin(B_VE + (2 * it + 1) % VS, (2 * it + 1) / VS + 1);
          const int z_end = (n_nodes + 31) & ~31;       // V rows up to the 32-token step: zeros
          for (int e = tid; e < (z_end - n_nodes) * (D / 16) * 2; e += 256) {
            const int t = e / (z_end - n_nodes), r = n_nodes + e % (z_end - n_nodes);
            const int h = t & 1, c16 = t >> 1;
            *reinterpret_cast<uint4*>(sV + (2 * it + h) % VS * K::kHalf + (r >> 3) * K::kGroupBytes + (c16 >> 3) * 1024 +
                                      (r & 7) * 128 + (((c16 & 7) ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
          }
        }
        for (int base = warp * RPW; base < n_stage; base += 8 * RPW * U) {
          uint4 x[U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int r = base + i * 8 * RPW + sub;
            const __nv_bfloat16* src = nullptr;
            if (r < rows) src = p.q + (long long)(q0 + r / hpc) * p.q_stride + (head0 + r % hpc) * D;
            else if (r >= n_q && r < n_q + n_draft) src = p.k_new + (long long)(q0 + r - n_q) * p.k_stride + pc.g * D;
            else if (r >= n_q && r < n_stage) src = p.v_new + (long long)(q0 + r - n_q - n_draft) * p.v_stride + pc.g * D;
            x[i] = src != nullptr ? __ldg(reinterpret_cast<const uint4*>(src) + ch) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int r = base + i * 8 * RPW + sub;
            uint32_t a = amax_bits(x[i]);
#pragma unroll
            for (int d = LPR / 2; d >= 1; d >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
            const bool wild = a >= 0x7f80u;             // a NaN or an infinity: zeros, and a NaN scale
            if (wild) { x[i] = make_uint4(0, 0, 0, 0); a = 0; }
            const int e = exp_of(a);
            uint2 hi, lo;
            split8(x[i], exp2i(-e), hi, lo);
            const float s = wild ? __int_as_float(0x7fc00000) : exp2i(e);
            const uint32_t in_row = (uint32_t)((((ch >> 1) & 7) << 4) | ((ch & 1) << 3));   // before the swizzle
            if (r < n_q) {
              uint8_t* at = sQ + (ch >> 4) * NQ * 128 + r * 128 + (in_row ^ ((r & 7) << 4));
              *reinterpret_cast<uint2*>(at) = hi;
              *reinterpret_cast<uint2*>(at + K::kQTerm) = lo;
              if (ch == 0) {
                sm->f[r] = s * p.scale * (MOD && p.softcap > 0.f ? 2.f * kLog2e / p.softcap : kLog2e);
                sm->m[r] = kNone;
                if (MOD) sm->slope[r] = p.slopes != nullptr && r < rows ? p.slopes[head0 + r % hpc] * kLog2e : 0.f;
              }
            } else if (r < n_stage) {
              const bool is_v = r >= n_q + n_draft;
              const int t = r - n_q - (is_v ? n_draft : 0);
              const uint32_t off = (uint32_t)((t >> 3) * K::kGroupBytes + (ch >> 4) * 1024 + (t & 7) * 128) + (in_row ^ ((t & 7) << 4));
              uint8_t* d_hi = is_v ? sV + 2 * it % VS * K::kHalf : sK + it % KS * K::kTileBytes;
              uint8_t* d_lo = is_v ? sV + (2 * it + 1) % VS * K::kHalf : d_hi + 8 * K::kGroupBytes;
              *reinterpret_cast<uint2*>(d_hi + off) = hi;
              *reinterpret_cast<uint2*>(d_lo + off) = lo;
              if (ch == 0) (is_v ? sm->row_v : sm->row_k)[t] = s;
            }
          }
        }
      }
      fence_async_smem();
      if (!sync_all()) break;
      // the tree: root paths and depths
      if (tid < n_nodes) {
        unsigned long long a = 1ull << tid;
        int d = 0;
        bool good = sm->par[tid] >= -1 && (tid > 0 || sm->par[0] == -1);
        for (int v = tid; good && v > 0; ++d) {
          const int up = sm->par[v];
          good = up >= 0 && up < v;
          if (good) a |= 1ull << up;
          v = up;
        }
        if (!good) {
          report(p.dev_status, SD_DEV_BAD_PARENTS);
          a = 1ull << tid;
          d = 0;
        }
        sm->anc[tid] = a;
        sm->depth[tid] = d;
        if (has_draft && sm->row_v[tid] != sm->row_v[tid]) sm->row_k[tid] = sm->row_v[tid];   // NaN: to the scores
      }
      if (!sync_all()) break;
      if (MOD) {
        for (int q = tid; q < nc * 16; q += 256) sm->dep[q] = q < rows ? (float)sm->depth[q / hpc] : 0.f;
        if (!sync_all()) break;
      }
      if (tid == 0) {
        mbar_arrive(bar(B_Q));
        if (has_draft) {
          mbar_arrive(bar(B_KF + it % KS));
          mbar_arrive(bar(B_VF + 2 * it % VS));
          mbar_arrive(bar(B_VF + (2 * it + 1) % VS));
        }
      }

      float2 sum[HC][8];
#pragma unroll
      for (int c = 0; c < HC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[c][e] = make_float2(0.f, 0.f);
      const int lo_root = p.window > 0 ? pc.L - p.window + 1 : 0;

      for (int i = 0; i < pc.tiles; ++i, ++it) {
        const bool draft = pc.first + i == 0;
        const int t0 = pc.base + (pc.first + i - 1) * kTile;
        const int valid = draft ? n_nodes : min(kTile, pc.L - t0);
        const bool band = !draft && p.window > 0 && t0 < lo_root + kMaxNodes;
        const bool masked = draft || valid < kTile || band;
        float ks = 1.f, vs = 1.f;
        if (draft) {
          if (row < n_nodes) { ks = sm->row_k[row]; vs = sm->row_v[row]; if (vs != vs) vs = 1.f; }
        } else {
          ok = spin(B_SC + it % SC, it / SC);
          if (!ok) break;
          ks = sm->scale[it % SC][row >> 4];
          vs = sm->scale[it % SC][8 + (row >> 4)];
          if (band && t0 + row >= lo_root && t0 + row < min(pc.L, lo_root + kMaxNodes)) {
            // a token that a window may hide from some nodes: its NaN codes of V become NaN scores
            const int pg = p.page_table[(size_t)pc.b * p.max_pages + (t0 + row) / kPage];
            if (pg >= 0 && pg < p.num_pool_pages) {
              const uint4* src = reinterpret_cast<const uint4*>(
                  p.v_cache + (((size_t)pg * p.hkv + pc.g) * kPage + (t0 + row) % kPage) * D);
              uint32_t nan = 0;
              for (int e = 0; e < D / 16; ++e) {
                const uint4 v = __ldg(src + e);
                nan |= __vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                       __vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
              }
              if (nan != 0u) ks = __int_as_float(0x7fc00000);
            }
          }
        }
        // Which of this thread's columns see its token row: one bit per column of the half.
        constexpr int VW = (HC * 16 + 31) / 32;
        uint32_t vis[VW];
#pragma unroll
        for (int w = 0; w < VW; ++w) vis[w] = row < valid ? 0xffffffffu : 0u;
        if (draft || band) {
          const int pos = t0 + row;
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            uint32_t bits = 0u;
#pragma unroll 1
            for (int e = 0; e < 32; ++e) {
              const int q = col0 + w * 32 + e;
              if (w * 32 + e >= mine * 16) break;
              const int dq = q < rows ? sm->depth[q / hpc] : 0;
              bool see = true;
              if (draft) {
                const int node = q < rows ? q / hpc : 0;
                see = row < n_nodes && ((sm->anc[node] >> row) & 1ull);
                if (p.window > 0 && see) see = dq - sm->depth[row] < p.window;
              } else {
                see = pos >= lo_root + dq;
              }
              bits |= (see ? 1u : 0u) << e;
            }
            vis[w] &= bits;
          }
        }
        const float rel = draft ? (row < n_nodes ? (float)sm->depth[row] : 0.f) : (float)(t0 + row - pc.L);
        ok = spin(B_SF + it % NS, it / NS);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_addr = tmem + lane_addr + (it % NS) * NQ + col0;
        uint32_t hi[HC][4], lo[HC][4];
        // base-2 score of a column pair from the raw product
        auto score2 = [&](float2 a, float2 f, int q) -> float2 {
          float2 s = mul2(a, mul2(f, make_float2(ks, ks)));
          if (MOD) {
            if (p.softcap > 0.f) {
              // c tanh(x / c) = c - 2 c / (1 + 2^(2 log2e x / c)); f holds the factor of the exponent
              const float cl = p.softcap * kLog2e;
              s.x = fmaf(-2.f * cl, fast_rcp(1.f + fast_exp2(s.x)), cl);
              s.y = fmaf(-2.f * cl, fast_rcp(1.f + fast_exp2(s.y)), cl);
            }
            if (p.slopes != nullptr) {
              s.x = fmaf(sm->slope[q], rel - sm->dep[q], s.x);
              s.y = fmaf(sm->slope[q + 1], rel - sm->dep[q + 1], s.y);
            }
          }
          return s;
        };
        uint32_t added = 0;      // chunks whose weights are in `sum` already
        bool over = i == 0 || masked;
        if (!over) {
          // One pass with the reference as it stands.
#pragma unroll
          for (int c = 0; c < HC; ++c) {
            if (c < mine) {
              float a[16];
              tmem_ld16(s_addr + c * 16, a);
              tmem_wait_ld();
              const int q = col0 + c * 16;
              float2 w[8];
              float top = 0.f;
              float2 e2[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 f = *reinterpret_cast<const float2*>(&sm->f[q + 2 * e]);
                const float2 m = *reinterpret_cast<const float2*>(&sm->m[q + 2 * e]);
                float2 d;
                if (MOD) {
                  const float2 s = score2(make_float2(a[2 * e], a[2 * e + 1]), f, q + 2 * e);
                  d = make_float2(s.x - m.x, s.y - m.y);
                } else {
                  d = fma2(make_float2(a[2 * e], a[2 * e + 1]), mul2(f, make_float2(ks, ks)), make_float2(-m.x, -m.y));
                }
                e2[e] = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                w[e] = mul2(e2[e], make_float2(vs, vs));
                top = fmaxf(top, fmaxf(w[e].x, w[e].y));
              }
              if (__any_sync(0xffffffffu, top > kTop)) {
                over = true;
              } else {
                added |= 1u << c;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[c][e] = add2(sum[c][e], e2[e]);
#pragma unroll
                for (int k = 0; k < 4; ++k) split4(w[2 * k], w[2 * k + 1], hi[c][k], lo[c][k]);
              }
            }
          }
          if (lane == 0) sm->flag[half][it & 1][quarter] = over ? 1 : 0;
          ok = sync_half();
          if (!ok) break;
          const int* fl = sm->flag[half][it & 1];
          over = (fl[0] | fl[1] | fl[2] | fl[3]) != 0;
        }
        if (over) {
          // The exact maxima of this tile, new references and rescale factors, then the weights.
          const float lv = fast_log2(vs);
#pragma unroll
          for (int c = 0; c < HC; ++c) {
            if (c < mine) {
              float a[16];
              tmem_ld16(s_addr + c * 16, a);
              tmem_wait_ld();
              const int q = col0 + c * 16;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 s = score2(make_float2(a[2 * e], a[2 * e + 1]), *reinterpret_cast<const float2*>(&sm->f[q + 2 * e]), q + 2 * e);
                const uint32_t v = vis[c / 2] >> ((c & 1) * 16 + 2 * e);
                a[2 * e] = v & 1u ? s.x + lv : -INFINITY;
                a[2 * e + 1] = v & 2u ? s.y + lv : -INFINITY;
              }
              const float mx = reduce16<true>(a, lane);
              if (lane < 16) sm->red[quarter][q + lane] = mx;
            }
          }
          ok = sync_half();
          if (!ok) break;
          const int q = col0 + quarter * 32 + lane;
          if (quarter * 32 + lane < mine * 16) {
            const float mt = fmaxf(fmaxf(sm->red[0][q], sm->red[1][q]), fmaxf(sm->red[2][q], sm->red[3][q]));
            const float old = sm->m[q], now = fmaxf(old, mt - kHead);
            sm->alpha[q] = fast_exp2(old - now);
            sm->m[q] = now;
          }
          ok = sync_half();
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < HC; ++c) {
            if (c < mine) {
              float a[16];
              tmem_ld16(s_addr + c * 16, a);
              tmem_wait_ld();
              const int qc = col0 + c * 16;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float2 w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int e = 2 * k + h;
                  const float2 s = score2(make_float2(a[2 * e], a[2 * e + 1]), *reinterpret_cast<const float2*>(&sm->f[qc + 2 * e]), qc + 2 * e);
                  const float2 m = *reinterpret_cast<const float2*>(&sm->m[qc + 2 * e]);
                  const float2 al = *reinterpret_cast<const float2*>(&sm->alpha[qc + 2 * e]);
                  const uint32_t v = vis[c / 2] >> ((c & 1) * 16 + 2 * e);
                  float2 ex;
                  ex.x = v & 1u ? fast_exp2(s.x - m.x) : 0.f;
                  ex.y = v & 2u ? fast_exp2(s.y - m.y) : 0.f;
                  sum[c][e] = mul2(sum[c][e], al);
                  if (!((added >> c) & 1u)) sum[c][e] = add2(sum[c][e], ex);
                  w[h].x = v & 1u ? ex.x * vs : 0.f;
                  w[h].y = v & 2u ? ex.y * vs : 0.f;
                }
                split4(w[0], w[1], hi[c][k], lo[c][k]);
              }
            }
          }
        }
        // S is read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_SE + it % NS));
        // P and O belong to the previous tile's PV until it has finished
        if (it > 0) {
          ok = spin(B_OD, it - 1);
          if (!ok) break;
        }
        tc_fence_after();
        if (over && i > 0) {
#pragma unroll 1
          for (int mb = 0; mb < MH; ++mb) {
#pragma unroll 1
            for (int c = 0; c < mine; ++c) {
              float v[16];
              const uint32_t ad = tmem + lane_addr + kColO + mb * NQ + col0 + c * 16;
              tmem_ld16(ad, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] *= sm->alpha[col0 + c * 16 + e];
              tmem_st16(ad, v);
            }
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          if (c < mine) {
            uint8_t* at = sP + (c_first + c) * kTile * 16 + row * 16;
            *reinterpret_cast<uint4*>(at) = make_uint4(hi[c][0], hi[c][1], hi[c][2], hi[c][3]);
            *reinterpret_cast<uint4*>(at + K::kPTerm) = make_uint4(lo[c][0], lo[c][1], lo[c][2], lo[c][3]);
          }
        }
        tc_fence_before();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PF));
      }
      if (!ok) break;

      // ---------------------------------------------------------- results
      // Column sums over the tile's 128 token rows: the lanes, then the quarters.
#pragma unroll
      for (int c = 0; c < HC; ++c) {
        if (c < mine) {
          float v[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) { v[2 * e] = sum[c][e].x; v[2 * e + 1] = sum[c][e].y; }
          const float s = reduce16<false>(v, lane);
          if (lane < 16) sm->red[quarter][col0 + c * 16 + lane] = s;
        }
      }
      ok = sync_half() && spin(B_OD, it - 1);
      if (!ok) break;
      tc_fence_after();
      const size_t slot = (size_t)blockIdx.x + pc.seg;      // rises by at least one along the pieces: unique
      {
        const int q = col0 + quarter * 32 + lane;
        if (quarter * 32 + lane < mine * 16) {
          const float l = sm->red[0][q] + sm->red[1][q] + sm->red[2][q] + sm->red[3][q];
          sm->alpha[q] = l == 0.f ? 0.f : 1.f / l;
          if (q < rows) {
            const float lse2 = l == 0.f ? -INFINITY : sm->m[q] + fast_log2(l);
            if (!pc.whole) p.lse_part[slot * NQ + q] = lse2;
            else if (p.lse != nullptr) p.lse[(size_t)(q0 + q / hpc) * p.hq + head0 + q % hpc] = lse2 * kLn2;
          }
        }
      }
      ok = sync_half();
      if (!ok) break;
      const bool odd = lane & 1;
#pragma unroll 1
      for (int c = 0; c < mine; ++c) {
#pragma unroll
        for (int mb = 0; mb < MH; ++mb) {
          float v[16];
          tmem_ld16(tmem + lane_addr + kColO + mb * NQ + col0 + c * 16, v);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int qe = col0 + c * 16 + 2 * k;
            const float ev = v[2 * k] * sm->alpha[qe], od = v[2 * k + 1] * sm->alpha[qe + 1];
            // even lanes keep the even column and take the odd lane's dim of it; odd lanes the reverse
            const float got = __shfl_xor_sync(0xffffffffu, odd ? ev : od, 1);
            const __nv_bfloat162 h = __floats2bfloat162_rn(odd ? got : ev, odd ? od : got);
            const int q = qe + (odd ? 1 : 0);
            if (q < rows) {
              __nv_bfloat16* dst = pc.whole ? p.out + ((size_t)(q0 + q / hpc) * p.hq + head0 + q % hpc) * D
                                            : p.o_part + (slot * NQ + q) * D;
              *reinterpret_cast<__nv_bfloat162*>(dst + mb * 128 + (row & ~1)) = h;
            }
          }
        }
      }
      tc_fence_before();
      // every warp is done with the columns' arrays and O before the next piece is staged
      ok = sync_all();
      tc_fence_after();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpQK) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(K::kTmem));
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace
}  // namespace sdv
