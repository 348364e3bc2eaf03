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
// less a few bits: the largest weight e c_t stays near 1 however uneven the
// blocks are (a token of the same e in a block of far smaller scale has a small
// weight), and m moves (with O and l rescaled) only when a weight passes kTop,
// the largest e4m3 value.
//
// The 8-bit operands.  K and V are exact as they lie.  A bf16 query is two
// e4m3 terms (a power-of-two scale for each query, which its column's scores
// take back in fp32, then the rounded value and the rounded rest: off by at
// most half of e4m3's smallest step, 2^-10 of an amax of 224 to 448, so by less
// than 2^-17 of the query's own amax);
// both multiply the same K tile into the same accumulator.  A weight is an
// e4m3 term and an e5m2 rest (2^-4 times 2^-3: at most 2^-7 off, about 2^-9.5
// in the mean square, while the term is normal; e5m2 so that the rest of small
// weights keeps its exponent range, down to 2^-16).  l sums the unrounded fp32 weights.  Draft
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
// host knowledge of the lengths.  Where every segment can have CTAs of its own
// for at most an eighth more units per CTA, it does (a second piece costs a CTA
// another staging and epilogue); else the line is cut where it falls, and no CTA
// idles on a ragged batch.  A segment in several pieces leaves fp32 partial
// outputs and log-sum-exps for the merge (bf16 ones are off by 2^-9 each: a typical
// error of 0.0025 of the outputs instead of 0.0019, and 0 to 1 us less for a call;
// f16 ones with a scale per column and quarter of the dims cost their maxima what
// they save); one in a single piece is written directly.  Context tiles go from the last to the first: a bias that falls with
// distance then has its largest scores first, and m moves once.
//
// Per tile (tokens are the MMA's M; NQ columns):
//   S[128 tok][NQ]     = K_tile . (Qhi + Qlo)^T      K-major, K = 32 a step
//   O^T[D][NQ]        += V_tile^T . (Phi + Plo)^T    M = 128 dims a product, MN-major
// Warps: NG groups of four softmax warps (lane quarter = warp % 4, a share of the
// columns per group; thread = token row), which also stage Q and the draft block
// and write the results; then one warp each that loads K and the block scales,
// loads V, issues QK, issues PV.
// Measured (one GB300).  A tile costs an SM, 256 dims: 1.42 us up to 48 columns
// (HBM: 7 TB/s of reads over 152 SMs), 2.04 at 96, 2.53 at 144, where its bytes
// would take 1.4, its products 1.25 (75 cycles each) and the softmax warps issue in
// 43 % of their slots; 128 dims: 0.75 at 16, 1.12 at 48, 1.65 at 96, 2.09 at 144.
// A call costs 9 us beyond its tiles at 16 columns, 11 to 12 up to 48 and 14 to 22
// beyond (plan 1.5, staging 3 to 6, the first references 2, results 1 to 4, the
// merge 3 to 5).  64 sequences of 1 to 32768 tokens, single tokens, 128 dims: 393 us,
// 6.4 TB/s; a tree of 23 over 131072 tokens, 256 dims: 89 us, 3.0 TB/s.  Of that, the
// queries' own scales (one multiplication a score) are 1.5 us and the small weights'
// rounding (see split4) 2.
// Every wait on a barrier is bounded; on expiry the kernel reports
// SD_DEV_TIMEOUT and runs out.
#pragma once

#include <cstddef>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace sdv {
namespace {

constexpr int kTile = kTileTokens;
constexpr float kTop = 448.0f;         // weights beyond it move m
// Where the largest weight so far sits after m moved: at 2^3 when m is set by a column's first tile, whose maximum is
// likely to be passed by some nats further on, at 2^5 when it was passed by so much that m had to move (a move costs a
// tile 2 us).  Lower means fewer moves, and coarser small weights: where the largest is 2^h, weights below 2^(-6 - h)
// of it keep an e5m2 value's bits, right in the mean of many alike (see split4), and those below 2^(-17 - h) nothing.  h
// grows with the piece, so that what is lost of its n tokens, n 2^(-17 - h), stays below 2^-7 of the largest weight up
// to 131072 of them.  At 2^1 and 2^2 a tree of 23 over 131072 tokens takes 83.6 us instead of 88.9, for limits four times
// as high.  (Tiles go from the last to the first and every piece has references of its own, so a peak at the front of a
// context hides none of it.)
constexpr float kHeadFirst = 3.0f, kHeadNext = 5.0f;
__device__ __forceinline__ float head_of(int tiles, bool first) {
  const float least = tiles > 256 ? 7.0f : tiles > 64 ? 5.0f : 3.0f;
  return fmaxf(least, first ? kHeadFirst : kHeadNext);
}
constexpr float kDown = 0x1p-8f;       // weights are formed times 2^-8 (see split4)
constexpr float kScaleLo = 0x1p-100f, kScaleHi = 0x1p100f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kScaleStages = 6;

// TIGHT: 144 columns of 256 dims leave 7 KB beside the operands and seven 16 KB half tiles.
template <int NQ, bool MOD, bool TIGHT>
struct KvSmall {
  static constexpr int kBars = TIGHT ? 24 : 40;
  float m[NQ];             // the column's reference, negated: -m
  float alpha[NQ];         // rescale factor of the current tile; 1 / l in the epilogue
  float qf[NQ];            // power-of-two scale of the column's query
  float slope[MOD ? NQ : 4];   // distance bias of the column, base 2
  float one[4];            // 1 in place of a query's scale, where the cap has taken it
  float red[4][NQ];        // per lane quarter: column maxima of a tile; column sums in the epilogue
  float scale[kScaleStages][16];   // K scales, then V scales, of a tile's eight pages
  float row_k[kMaxNodes], row_v[kMaxNodes];   // scales of the draft block's rows
  unsigned long long anc[kMaxNodes];          // bit r: node r is on the node's root path; in the draft CTA then turned
                                              // round, bit n: node n sees the row
  uint64_t bar[kBars];
  int cum[kMaxBatch + 1];  // first unit of each sequence
  int scan[8];
  int per, extra;
  int8_t par[kMaxNodes];
  int8_t depth[kMaxNodes];
  alignas(16) int flag[3][2][4];   // [group][tile parity][lane quarter]: chunks where a weight passes kTop
  uint32_t tmem;
  int abort;
};

// D: head dim.  NG groups of softmax warps, of up to CC 16-column chunks each.  MOD: capped scores or a distance bias.
template <int D, int NG, int CC, bool MOD>
struct Kv {
  static constexpr int NQ = NG * CC * 16;                 // query columns
  static constexpr int kWarps = NG * 4, kThreads = (kWarps + 4) * 32;
  using Small = KvSmall<NQ, MOD, NQ == 144 && D == 256>;
  // One group: a tile is a chain of short steps (scores, weights, products), and a second CTA on the SM fills its waits.
  static constexpr int kCtas = NG == 1 ? 2 : 1;
  static constexpr int kSmemBytes = kCtas == 2 ? 115712 : 232448;   // dynamic shared memory a CTA can have
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
  static constexpr int KS = kUnits < 6 ? 1 : kUnits < 8 ? 2 : kUnits / 4;   // K tiles
  static constexpr int VS = kUnits - 2 * KS;                   // V half tiles
  static constexpr size_t kSmem = (size_t)kQBytes + kPBytes + KS * kTileBytes + VS * kHalf + sizeof(Small);
  static_assert(VS >= 2, "the V ring holds a tile");
  static_assert(KS + NS <= kScaleStages, "scale stages");
  static_assert(kSmem <= (size_t)kSmemBytes, "shared memory over 227 KB");
};

// ------------------------------------------------------------ small pieces

// A bounded wait, kept short (every instruction of this kernel's loops comes through a small instruction cache):
// false, with the CTA's abort flag set, if the phase never completes.  The kernel's end reports the flag.
__device__ __forceinline__ bool wait8(uint32_t bar, uint32_t parity, volatile int* abort) {
  long long t0 = 0;
#pragma unroll 1
  while (!mbar_try(bar, parity)) {
    const long long now = clock64();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitCycles || *abort) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// One lane of a converged warp.  The tensor core's and TMA's instructions take uniform operands: issued by an elected
// lane of a warp that runs as one they cost a few instructions, issued under a plain lane test several dozen each.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ uint64_t noswz_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}
// kind::f8f6f4, fp32 accumulators: A e4m3, B e4m3 or e5m2.
__device__ __forceinline__ uint32_t f8_idesc(int n, int a_mn, int b_mn, bool b_e5m2) {
  return (1u << 4) | (b_e5m2 ? 1u << 10 : 0u) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// ACC: 0 overwrites D, 1 adds to it, 2 as `acc` says.  One lane issues some thirty of these per tile, so their
// operands are a descriptor plus a constant and nothing is decided at run time that need not be.
template <int ACC>
__device__ __forceinline__ void umma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc = 1) {
  if (ACC == 2)
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "n"(ACC));
}
__device__ __forceinline__ void tma_page8(uint32_t dst, const CUtensorMap* map, int w, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3}], [%4], %5;"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(w), "r"(bar), "l"(policy)
      : "memory");
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
// Four weights w (two pairs, columns in order, each times 2^-8) as four e4m3 codes and four e5m2 codes of the
// rest, w in [0, 448].  The 8-bit conversions share a slow pipe with exp2, so they are done on f16 bits: w * 2^-8
// has e4m3's exponent bias in f16, subnormals included, so the code is the rounded top byte below the sign; e5m2
// is the top byte of f16.  Both round half away (off by at most half a step, like any nearest rounding; a tie
// costs a weight nothing that its rest does not give back).  A NaN weight loses itself here and is carried by the
// column's sum.  Weights below 2^-6 have few bits left in the rest, and a long context has many alike, which a nearest
// rounding puts off by the same 2^-3 at most (8064 tokens 9.6 nats below a peak: 5.7 times 2^-7 of the output).  Their
// rests round up from a border of the token row's own instead, `spread` (see spread_of): off by a step of the rest each,
// but not in the mean of a tile's rows (0.4 times 2^-7; 0.97 where what falls below 2^-17 is counted in).
__device__ __forceinline__ uint32_t spread_of(int row) {
  // a 256th for each row, even over any 2^k aligned ones: the row's bits turned round.  What is added before a rest's low
  // byte is cut, against the 0x80 of a nearest rounding.
  const uint32_t add = (__brev((uint32_t)row) >> 25) * 2u + 1u;
  return (add ^ 0x80u) * 0x00010001u;
}
__device__ __forceinline__ void split4(float2 w0, float2 w1, uint32_t spread, uint32_t& hi, uint32_t& lo) {
  const __half2 a = __floats2half2_rn(w0.x, w0.y), b = __floats2half2_rn(w1.x, w1.y);
  const uint32_t ta = *reinterpret_cast<const uint32_t*>(&a) + 0x00400040u;
  const uint32_t tb = *reinterpret_cast<const uint32_t*>(&b) + 0x00400040u;
  hi = __byte_perm(ta >> 7, tb >> 7, 0x6420);
  const uint32_t ha = ta & 0x7f807f80u, hb = tb & 0x7f807f80u;
  const __half2 up = __halves2half2(__ushort_as_half(0x5c00), __ushort_as_half(0x5c00));   // 2^8
  const __half2 ra = __hmul2(__hsub2(a, *reinterpret_cast<const __half2*>(&ha)), up);
  const __half2 rb = __hmul2(__hsub2(b, *reinterpret_cast<const __half2*>(&hb)), up);
  const __half2 least = __halves2half2(__ushort_as_half(0x0400), __ushort_as_half(0x0400));   // 2^-14: a weight of 2^-6
  const uint32_t add_a = (__hlt2_mask(a, least) & spread) ^ 0x00800080u;
  const uint32_t add_b = (__hlt2_mask(b, least) & spread) ^ 0x00800080u;
  lo = __byte_perm(*reinterpret_cast<const uint32_t*>(&ra) + add_a, *reinterpret_cast<const uint32_t*>(&rb) + add_b, 0x7531);
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Maxima of 16 values (each lane's plus `plus`) over the warp's lanes: lane L ends with that of value L % 16.
__device__ __forceinline__ float warp_max16(const float (&v)[16], float plus, int lane) {
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(x) : "f"(v[i] + plus));
    r = (lane & 15) == i ? x : r;
  }
  return r;
}
// Sums of 16 values over the warp's lanes: lane L ends with that of value L % 16.
__device__ __forceinline__ float warp_sum16(float (&v)[16], int lane) {
#pragma unroll
  for (int half = 8; half >= 1; half >>= 1) {
    const bool up = (lane & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, half);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

// Eight bf16 as two e4m3 terms (hi + lo) of x * 2^-e.  In f16 on the way: 8 significant bits survive it wherever the
// two terms could hold them.
__device__ __forceinline__ uint32_t split2(uint32_t w, float inv) {   // hi pair below, lo pair above
  const float2 v = mul2(__bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w)), make_float2(inv, inv));
  uint32_t r;
  asm("{ .reg .b32 a, b; .reg .b16 s, t;\n\t"
      "cvt.rn.f16x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 s, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 b, s;\n\t"
      "sub.rn.f16x2 a, a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 t, a;\n\t"
      "mov.b32 %0, {s, t}; }"
      : "=r"(r)
      : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ void split8(const uint4 x, float inv, uint2& hi, uint2& lo) {
  const uint32_t a = split2(x.x, inv), b = split2(x.y, inv), c = split2(x.z, inv), d = split2(x.w, inv);
  hi = make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410));
  lo = make_uint2(__byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x7632));
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
// The same for a query, whose scale only its own scores meet: any bf16 amax (2^e and 2^-e are normal numbers).
__device__ __forceinline__ int query_exp(uint32_t bits) {
  return max(-126, (int)(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0));
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// What a segment's draft tile counts for beyond one unit, where CTAs have `even` units each: staging the block, its masks
// and the moves of fresh references take some 5 us, a tile of 144 columns 2.3 us and one of 96 or fewer 1.2 to 1.8; in
// pieces of few units one more would cost the whole.  Against 2 from 12 units and 1 from 5 on: a tree of 23 over 32768
// tokens 39.3 -> 37.8 us, 8 sequences of 8 nodes 38.5 -> 37.8 (128 dims), 16 nodes over 32768 31.7 -> 29.8.
template <int NQ>
__device__ __forceinline__ int extra_units(int even) {
  return even >= 12 && NQ < 144 ? 3 : even >= 6 ? 2 : even >= 4 ? 1 : 0;
}

// A bit per column of a softmax group.
template <int CC> struct BitsOf { using type = uint32_t; };
template <> struct BitsOf<3> { using type = unsigned long long; };

// One CTA's share of one segment.
struct Piece {
  int b, g, c;         // sequence, KV head, head part
  int seg;
  int L, base, nt;     // context length; first position the context tiles cover, and how many there are
  int first, tiles;    // first tile of the segment (0: the draft block, i: the i-th context tile from the end), how many
  int span;            // units of the line that the piece takes
  bool whole;          // the segment lies in this piece alone
  __device__ __forceinline__ int t0(int i) const { return base + (nt - i) * kTile; }   // position of context tile i
};

template <int D, int NG, int CC, bool MOD>
__global__ void __launch_bounds__((NG + 1) * 128, NG == 1 ? 2 : 1)
kv8_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const Kv8AttnParams p, const BatchDesc bd) {
  using K = Kv<D, NG, CC, MOD>;
  constexpr int NQ = K::NQ, MH = K::MH, NS = K::NS, KS = K::KS, VS = K::VS;
  constexpr int kWarps = K::kWarps, kKvThreads = K::kThreads;      // softmax warps; all threads
  constexpr int kWarpK = kWarps, kWarpV = kWarps + 1, kWarpQK = kWarps + 2;
  using Sm = typename K::Small;
  constexpr int B_KF = 0, B_KE = KS, B_VF = 2 * KS, B_VE = B_VF + VS, B_SC = B_VE + VS, B_SF = B_SC + KS + NS,
                B_SE = B_SF + NS, B_PF = B_SE + NS, B_OD = B_PF + 1, B_Q = B_PF + 2, B_G = B_PF + 3;
  constexpr int kNumBars = B_G + NG;
  static_assert(kNumBars <= Sm::kBars, "barriers");
  constexpr int SC = KS + NS;   // scale stages: see the K producer
  extern __shared__ __align__(1024) uint8_t smem8[];
  uint8_t* sQ = smem8;
  uint8_t* sK = sQ + K::kQBytes;
  uint8_t* sV = sK + KS * K::kTileBytes;
  uint8_t* sP = sV + VS * K::kHalf;
  Sm* sm = reinterpret_cast<Sm*>(sP + K::kPBytes);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (smem_u32(smem8) & 1023u) {   // not expected; refuse rather than mis-swizzle
    if (tid == 0) report_dep(p.dev_status, SD_DEV_TIMEOUT);
    return;
  }

  // ---------------------------------------------------------------- the line of units
  const int parts = p.hkv * p.hparts;   // segments per sequence
  auto ctx_of = [&](int b) {
    const int L = p.ctx_lens[b];
    return L < 0 ? 0 : min(L, p.max_pages * kPage);
  };
  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(smem_u32(&sm->bar[i]), i == B_PF || (i >= B_SE && i < B_SE + NS) ? (uint32_t)kWarps : i >= B_G ? 4u : 1u);
    sm->abort = 0;
    sm->one[0] = sm->one[1] = sm->one[2] = sm->one[3] = 1.f;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Launched as a programmatic dependent: everything above touches no global memory; here the previous kernel's writes
  // become visible.  The merge's blocks may be scheduled as this kernel's CTAs leave.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (bd.batch <= 32) {
    int per, extra;
    // a sequence per lane, every warp for itself
    int units = 0;
    if (lane < bd.batch) {
      const int raw = p.ctx_lens[lane], L = ctx_of(lane);
      if (blockIdx.x == 0 && warp == 0 && raw != L) report(p.dev_status, SD_DEV_BAD_CTX);
      units = 1 + (L - window_base(L, p.window, kTile) + kTile - 1) / kTile;
    }
    const int even = (__reduce_add_sync(0xffffffffu, units) * parts + (int)gridDim.x - 1) / (int)gridDim.x;
    const int more = extra_units<NQ>(even);
    per = even;
    extra = -1;
#pragma unroll 1
    for (int w = 0; w < 8 && extra < 0; ++w) {
      const int size = even + w * max(1, even / 56);
      const int need = __reduce_add_sync(0xffffffffu, units > 0 ? (units + more + size - 1) / size : 0) * parts;
      if (need <= (int)gridDim.x) { per = size; extra = more; }
    }
    int incl = (extra >= 0 ? (units + (units > 0 ? extra : 0) + per - 1) / per * per : units) * parts;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    if (warp == 0) {
      if (lane == 0) { sm->cum[0] = 0; sm->per = per; sm->extra = extra; }
      if (lane < bd.batch) sm->cum[lane + 1] = incl;
    }
  } else {
    int per, extra;
    int units = 0;
    if (tid < bd.batch) {
      const int raw = p.ctx_lens[tid], L = ctx_of(tid);
      if (blockIdx.x == 0 && raw != L) report(p.dev_status, SD_DEV_BAD_CTX);
      units = 1 + (L - window_base(L, p.window, kTile) + kTile - 1) / kTile;
      sm->cum[tid] = units;
    }
    __syncthreads();
    // Eight warps try eight piece sizes, from the even share up.
    if (warp < 8) {
      int sum = 0;
#pragma unroll 1
      for (int b = lane; b < bd.batch; b += 32) sum += sm->cum[b];
      sum = __reduce_add_sync(0xffffffffu, sum);
      const int even = (sum * parts + (int)gridDim.x - 1) / (int)gridDim.x;
      const int more = extra_units<NQ>(even);
      const int size = even + warp * max(1, even / 56);
      int need = 0;
#pragma unroll 1
      for (int b = lane; b < bd.batch; b += 32) need += (sm->cum[b] + more + size - 1) / size;
      need = __reduce_add_sync(0xffffffffu, need) * parts;
      if (lane == 0) sm->scan[warp] = need <= (int)gridDim.x ? size : 0;
      if (tid == 0) { sm->flag[0][0][0] = even; sm->flag[0][0][1] = more; }
    }
    __syncthreads();
    per = 0;
#pragma unroll
    for (int w = 7; w >= 0; --w) per = sm->scan[w] > 0 ? sm->scan[w] : per;
    extra = per > 0 ? sm->flag[0][0][1] : -1;
    if (per == 0) per = sm->flag[0][0][0];
    __syncthreads();
    int incl = (extra >= 0 ? (units + (units > 0 ? extra : 0) + per - 1) / per * per : units) * parts;
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
#pragma unroll 1
      for (int w = 0; w < warp; ++w) incl += sm->scan[w];
      if (tid == 0) { sm->cum[0] = 0; sm->per = per; sm->extra = extra; }
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
  // units per CTA; extra >= 0: every segment has CTAs of its own, its draft tile counting 1 + extra units
  const int per = sm->per, extra = sm->extra;
  const int total = sm->cum[bd.batch];
  const int u_begin = min(total, (int)blockIdx.x * per), u_end = min(total, u_begin + per);
  if (blockIdx.x == 0) {   // for the merge
#pragma unroll 1
    for (int i = tid; i <= bd.batch; i += kKvThreads) p.cum[i] = sm->cum[i];
    if (tid == 0) { p.cum[kMaxBatch + 1] = per; p.cum[kMaxBatch + 2] = extra; }
  }
  // The piece that begins at unit u.
  auto piece_at = [&](int u) {
    Piece pc;
    int lo = 0, hi = bd.batch - 1;
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sm->cum[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const int line = (sm->cum[lo + 1] - sm->cum[lo]) / parts;     // units of one of the sequence's segments
    const int rem = u - sm->cum[lo], s = rem / line, at = rem - s * line;
    pc.b = lo;
    pc.g = s / p.hparts;
    pc.c = s - pc.g * p.hparts;
    pc.seg = lo * parts + s;
    pc.L = ctx_of(lo);
    pc.base = window_base(pc.L, p.window, kTile);
    pc.nt = (pc.L - pc.base + kTile - 1) / kTile;
    if (extra >= 0) {
      pc.first = max(0, at - extra);
      pc.tiles = min(pc.nt + 1, at + per - extra) - pc.first;
      pc.span = per;
    } else {
      pc.first = at;
      pc.tiles = pc.span = min(line - at, u_end - u);
    }
    pc.whole = pc.tiles == pc.nt + 1;
    // the same for every lane, and known to be
    pc.b = __shfl_sync(0xffffffffu, pc.b, 0);
    pc.g = __shfl_sync(0xffffffffu, pc.g, 0);
    pc.c = __shfl_sync(0xffffffffu, pc.c, 0);
    pc.first = __shfl_sync(0xffffffffu, pc.first, 0);
    pc.tiles = __shfl_sync(0xffffffffu, pc.tiles, 0);
    pc.L = __shfl_sync(0xffffffffu, pc.L, 0);
    pc.base = __shfl_sync(0xffffffffu, pc.base, 0);
    pc.nt = __shfl_sync(0xffffffffu, pc.nt, 0);
    pc.span = __shfl_sync(0xffffffffu, pc.span, 0);
    return pc;
  };
  const uint32_t bars = smem_u32(&sm->bar[0]);
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto wait = [&](int i, int n) { return wait8(bar(i), (uint32_t)n & 1u, &sm->abort); };
  // The softmax warps do not leave early: after an expired wait no other one waits, and they run through, so that
  // their named barriers always find all of them.
  auto spin = [&](int i, int n) {
    wait(i, n);
    __syncwarp();
  };
  const uint32_t tmem = sm->tmem;
  const uint32_t kColO = NS * NQ;   // O^T behind the S buffers

  // Positions in the rings, counted along: an index and the parity of its round.
  struct Ring {
    int at = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next(int n) {
      if (++at == n) { at = 0; round ^= 1u; }
    }
  };
  auto wait_full = [&](int first, const Ring& r) { return wait(first + r.at, (int)r.round); };
  auto wait_empty = [&](int first, const Ring& r) { return wait(first + r.at, (int)r.round ^ 1); };

  // The softmax warps of the wider tiles need more registers than an even share: 3 x 152 + 56 is what the block was
  // launched with (4 x 128 per warp).
  constexpr bool kShare = NG > 1 && CC >= 2;
  if (warp >= kWarps) {
    if (kShare) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp <= kWarpV) {
      // ---------------------------------------------------------- producers
      // Page ids come a group of four tiles at a time (lane l: page l % 8 of the group's tile l / 8), two groups ahead of
      // their use, block scales one: under a full memory system a load takes as long as a tile or two.
      const bool is_k = warp == kWarpK;
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      const uint64_t policy = l2_evict_first();
      Ring ring, sc_ring;   // K tiles or V half tiles; scale stages
      bool ok = true;
#pragma unroll 1
      for (int u = u_begin; u < u_end && ok;) {
        const Piece pc = piece_at(u);
        u += pc.span;
        const int* row = p.page_table + (size_t)pc.b * p.max_pages;
        int left = pc.tiles;
        if (pc.first == 0) {
          // The draft tile is staged by the softmax warps: its slots, and its scale stage, pass by in their turn.  In
          // their turn means waiting for what they held before: a producer that went past a slot without that could
          // be two rounds ahead of it, which a barrier's parity cannot tell from none.  Nor may it fall two rounds
          // behind: the producers say that the slots are full as they come by, so that no product of a draft tile begins
          // before both have passed it (that its contents are there, B_Q and B_PF say).
          if (is_k) {
            ok = __all_sync(0xffffffffu, wait_empty(B_KE, ring));
            if (!ok) break;
            if (elect_one()) {
              mbar_arrive(bar(B_SC + sc_ring.at));
              mbar_arrive(bar(B_KF + ring.at));
            }
            __syncwarp();
            sc_ring.next(SC);
            ring.next(KS);
          } else {
#pragma unroll 1
            for (int h = 0; h < 2 && ok; ++h) {
              ok = __all_sync(0xffffffffu, wait_empty(B_VE, ring));
              if (ok && elect_one()) mbar_arrive(bar(B_VF + ring.at));
              __syncwarp();
              ring.next(VS);
            }
            if (!ok) break;
          }
          --left;
        }
        int t0 = pc.t0(max(pc.first, 1));
        auto ids_from = [&](int n) {     // of the piece's context tiles n .. n + 3
          const int t = t0 - (lane >> 3) * kTile + (lane & 7) * kPage;
          return n + (lane >> 3) < left && t - n * kTile < pc.L ? row[(t - n * kTile) / kPage] : -1;
        };
        auto in_pool = [&](int page) { return (unsigned)page < (unsigned)p.num_pool_pages; };
        auto scales_of = [&](const float* s, int page) {
          return is_k && in_pool(page) ? __ldg(s + (size_t)page * p.hkv + pc.g) : 1.f;
        };
        int ids_next = ids_from(0), ids_after = ids_from(4), ids = -1;
        float ks_next = scales_of(p.k_scales, ids_next), vs_next = scales_of(p.v_scales, ids_next), ks_now = 1.f, vs_now = 1.f;
        uint32_t good = 0;    // pages of the group that can be loaded
#pragma unroll 1
        for (int n = 0; n < left; ++n) {
          const int sub = (n & 3) * 8;
          if (sub == 0) {
            ids = ids_next;
            ks_now = ks_next;
            vs_now = vs_next;
            ids_next = ids_after;
            ids_after = ids_from(n + 8);
            ks_next = scales_of(p.k_scales, ids_next);
            vs_next = scales_of(p.v_scales, ids_next);
            good = __ballot_sync(0xffffffffu, in_pool(ids));
            if (is_k) {
              const int at = t0 - (n + (lane >> 3)) * kTile + (lane & 7) * kPage;
              if (n + (lane >> 3) < left && at < pc.L && !in_pool(ids)) report(p.dev_status, SD_DEV_BAD_PAGE);
              if (!(ks_now >= kScaleLo && ks_now <= kScaleHi && vs_now >= kScaleLo && vs_now <= kScaleHi)) {
                report(p.dev_status, SD_DEV_BAD_SCALE);
                ks_now = ks_now > kScaleHi ? kScaleHi : ks_now >= kScaleLo ? ks_now : kScaleLo;
                vs_now = vs_now > kScaleHi ? kScaleHi : vs_now >= kScaleLo ? vs_now : kScaleLo;
              }
            }
          }
          const uint32_t have = (good >> sub) & 0xffu;
          const int tile = t0 - n * kTile;
          const int valid = min(kTile, pc.L - tile);
          const uint32_t need = (1u << ((valid + kPage - 1) / kPage)) - 1u;
          const int half_page = (ids * p.hkv + pc.g) * 2;   // the tensor map's outer coordinate
          if (is_k) {
            ok = __all_sync(0xffffffffu, wait_empty(B_KE, ring));
            if (!ok) break;
            uint8_t* dst = sK + ring.at * K::kTileBytes;
            if (need & ~have) {   // ids out of range count as zeros (they cannot be read)
#pragma unroll 1
              for (int e = lane; e < 8 * (K::kPageBytes / 16); e += 32)
                if (((need & ~have) >> (e / (K::kPageBytes / 16))) & 1u)
                  reinterpret_cast<uint4*>(dst)[e] = make_uint4(0, 0, 0, 0);
              fence_async_smem();
              __syncwarp();
            }
            int w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __shfl_sync(0xffffffffu, half_page, sub + j);
            if (elect_one()) {
              mbar_expect_tx(bar(B_KF + ring.at), (uint32_t)__popc(have) * (uint32_t)K::kPageBytes);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if ((have >> j) & 1u) tma_page8(smem_u32(dst) + j * K::kPageBytes, map, w[j], bar(B_KF + ring.at), policy);
            }
            // A scale stage may be rewritten once the softmax has read the scores of the tile KS + NS before, which the
            // wait on K_EMPTY implies (that tile's successor by NS has been multiplied).
            const float k_sc = __shfl_sync(0xffffffffu, ks_now, sub + (lane & 7));
            const float v_sc = __shfl_sync(0xffffffffu, vs_now, sub + (lane & 7));
            if (lane < 16) sm->scale[sc_ring.at][lane] = lane < 8 ? k_sc : v_sc;
            __syncwarp();
            if (elect_one()) mbar_arrive(bar(B_SC + sc_ring.at));
            sc_ring.next(SC);
            ring.next(KS);
          } else {
            // V: two halves of 64 tokens, issued together where the ring holds two tiles.  Rows that nobody sees must be
            // zeros, not whatever lies there (a weight of 0 times a NaN code is NaN): pages with such rows, and those
            // that only some nodes of a tree see through a window, go through plain loads, the rest by TMA.
            constexpr int kJoint = VS >= 4 ? 2 : 1;
            const int lo = p.window > 0 ? pc.L - p.window + 1 : 0;          // the root's oldest visible position
            const int seen = p.window > 0 ? lo + kMaxNodes : 0;             // from here on every node sees every token
            uint32_t fast = have, slow = 0;
            if (have != 0xffu || valid < kTile || tile < seen) {
              const int at = tile + lane * kPage;
              // pages up to the last 32-token step of their half
              const int steps = lane < 4 ? (min(64, valid) + 31) / 32 * 2 : (max(0, valid - 64) + 31) / 32 * 2;
              const bool used = lane < 8 && (lane & 3) < steps;
              const bool plain = used && (!((have >> lane) & 1u) || at + kPage > pc.L || at < seen);
              slow = __ballot_sync(0xffffffffu, plain);
              fast = __ballot_sync(0xffffffffu, used && !plain);
            }
            int w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __shfl_sync(0xffffffffu, half_page, sub + j);
#pragma unroll
            for (int h = 0; h < 2; h += kJoint) {
              Ring other = ring;
              other.next(VS);
              ok = wait_empty(B_VE, ring);
              if (kJoint == 2) ok = ok && wait_empty(B_VE, other);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              const uint32_t sel = kJoint == 2 ? 0xffu : 0xfu << (4 * h);
              uint8_t* base[2] = {sV + ring.at * K::kHalf, sV + (kJoint == 2 ? other.at : ring.at) * K::kHalf};
              if (slow & sel) {
#pragma unroll 1
                for (int e = lane; e < 8 * kPage * (D / 16); e += 32) {
                  const int pg = e / (kPage * (D / 16)), r = e / (D / 16) % kPage, ch = e % (D / 16);
                  const int id = __shfl_sync(0xffffffffu, ids, sub + pg);
                  if (!(((slow & sel) >> pg) & 1u)) continue;
                  const int t = tile + pg * kPage + r;
                  uint4 v = make_uint4(0, 0, 0, 0);
                  if (in_pool(id) && t >= lo && t < pc.L) {
                    v = __ldg(reinterpret_cast<const uint4*>(p.v_cache + (((size_t)id * p.hkv + pc.g) * kPage + r) * D) + ch);
                    if (t < seen) {   // NaN codes: the softmax makes the row's scores NaN instead
                      uint32_t* x = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                      for (int k = 0; k < 4; ++k) x[k] &= ~__vcmpeq4(x[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    }
                  }
                  *reinterpret_cast<uint4*>((pg < 4 ? base[0] : base[1]) + (pg & 3) * K::kPageBytes +
                                            (r >> 3) * K::kGroupBytes + (ch >> 3) * 1024 + (r & 7) * 128 +
                                            (((ch & 7) ^ (r & 7)) << 4)) = v;
                }
                fence_async_smem();
                __syncwarp();
              }
              if (elect_one()) {
#pragma unroll
                for (int hh = h; hh < h + kJoint; ++hh) {
                  const uint32_t full = bar(B_VF + (hh > h ? other.at : ring.at));
                  const uint32_t mine = (fast >> (4 * hh)) & 0xfu;
                  mbar_expect_tx(full, (uint32_t)__popc(mine) * (uint32_t)K::kPageBytes);
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if ((mine >> j) & 1u)
                      tma_page8(smem_u32(base[hh > h ? 1 : 0]) + j * K::kPageBytes, map, w[4 * hh + j], full, policy);
                }
              }
              __syncwarp();
              for (int k = 0; k < kJoint; ++k) ring.next(VS);
            }
            if (!ok) break;
          }
        }
      }
      // After an abort no copy may still be landing when the CTA ends: wait, bounded, for both rounds of every slot.
      if (lane == 0 && *(volatile int*)&sm->abort) {
#pragma unroll 1
        for (int s = 0; s < 2 * (is_k ? KS : VS); ++s) {
          const long long begin = clock64();
          while (!mbar_test(bar((is_k ? B_KF : B_VF) + (s >> 1)), (uint32_t)s & 1u) && clock64() - begin < kWaitCycles / 64) {
          }
        }
      }
    } else if (warp == kWarpQK) {
      // ---------------------------------------------------------- QK issuer
      Ring s_ring, k_ring;
      int np = 0;
      bool ok = true;
      const uint64_t q_desc = sw128_desc(smem_u32(sQ), 16, 1024);
#pragma unroll 1
      for (int u = u_begin; u < u_end && ok; ++np) {
        const Piece pc = piece_at(u);
        u += pc.span;
        const int n_nodes = bd.q_indptr[pc.b + 1] - bd.q_indptr[pc.b];
        const int nq = (min(p.hpc, p.group - pc.c * p.hpc) * n_nodes + 15) & ~15;
        const uint32_t idesc = f8_idesc(nq, 0, 0, false);
        ok = __all_sync(0xffffffffu, wait(B_Q, np));
#pragma unroll 1
        for (int i = 0; i < pc.tiles && ok; ++i) {
          ok = wait_empty(B_SE, s_ring) && wait_full(B_KF, k_ring);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a0 = sw128_desc(smem_u32(sK + k_ring.at * K::kTileBytes), 16, K::kGroupBytes);
          const uint32_t d = tmem + s_ring.at * NQ;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              const uint64_t a = a0 + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4);
              const uint64_t b = q_desc + (((kk >> 2) * NQ * 128 + (kk & 3) * 32) >> 4);
              if (kk == 0) umma8<0>(d, a, b, idesc); else umma8<1>(d, a, b, idesc);
              umma8<1>(d, a, b + (K::kQTerm >> 4), idesc);
            }
            // The draft block: rows 0-63 hold the keys' first terms, rows 64-127 the second; both go to rows 0-63 of S
            // (its other rows then hold nothing and are masked).
            if (pc.first + i == 0) {
#pragma unroll 1
              for (int kk = 0; kk < D / 32; ++kk) {
                const uint32_t off = (kk & 3) * 32;
                const uint64_t a = a0 + ((8 * K::kGroupBytes + (kk >> 2) * 1024 + off) >> 4);
                const uint64_t b = q_desc + (((kk >> 2) * NQ * 128 + off) >> 4);
                umma8<1>(d, a, b, idesc);
                umma8<1>(d, a, b + (K::kQTerm >> 4), idesc);
              }
            }
            umma_commit(bar(B_KE + k_ring.at));
            umma_commit(bar(B_SF + s_ring.at));
          }
          __syncwarp();
          s_ring.next(NS);
          k_ring.next(KS);
        }
      }
    } else {
      // ---------------------------------------------------------- PV issuer
      Ring v_ring;
      int it = 0;
      bool ok = true;
      // P: 16-column chunks of 128 token rows x 16 bytes; MN-major without a swizzle
      const uint64_t p_desc = noswz_desc(smem_u32(sP), 128, kTile * 16);
#pragma unroll 1
      for (int u = u_begin; u < u_end && ok;) {
        const Piece pc = piece_at(u);
        u += pc.span;
        const int n_nodes = bd.q_indptr[pc.b + 1] - bd.q_indptr[pc.b];
        const int nq = (min(p.hpc, p.group - pc.c * p.hpc) * n_nodes + 15) & ~15;
        const uint32_t id_hi = f8_idesc(nq, 1, 1, false), id_lo = f8_idesc(nq, 1, 1, true);
#pragma unroll 1
        for (int i = 0; i < pc.tiles && ok; ++i, ++it) {
          const bool draft = pc.first + i == 0;
          const int valid = draft ? n_nodes : min(kTile, pc.L - pc.t0(pc.first + i));
          ok = __all_sync(0xffffffffu, wait(B_PF, it));
#pragma unroll 1
          for (int h = 0; h < 2 && ok; ++h) {
            ok = __all_sync(0xffffffffu, wait_full(B_VF, v_ring));
            if (!ok) break;
            tc_fence_after();
            // the draft block: half 0 the values' first terms, half 1 the second, both weighed by rows 0-63 of P
            const int rows = draft ? valid : valid - h * 64;
            const uint64_t v0 = sw128_desc(smem_u32(sV + v_ring.at * K::kHalf), 1024, K::kGroupBytes);
            const uint64_t p0 = p_desc + (draft ? 0 : (h * 64 * 16) >> 4);
            if (elect_one()) {
              // two 32-token steps: the weights' first term and their rest on each 128-dim block
#pragma unroll
              for (int ks = 0; ks < 2; ++ks) {
                if (rows > ks * 32) {
#pragma unroll
                  for (int mb = 0; mb < MH; ++mb) {
                    const uint64_t a = v0 + ((ks * 4 * K::kGroupBytes + mb * 1024) >> 4);
                    const uint64_t b = p0 + ((ks * 512) >> 4);
                    umma8<2>(tmem + kColO + mb * NQ, a, b, id_hi, i > 0 || h > 0 || ks > 0 ? 1u : 0u);
                    umma8<1>(tmem + kColO + mb * NQ, a, b + (K::kPTerm >> 4), id_lo);
                  }
                }
              }
              umma_commit(bar(B_VE + v_ring.at));
              if (h == 1) umma_commit(bar(B_OD));
            }
            __syncwarp();
            v_ring.next(VS);
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warps
    if (kShare) asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    const int group = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;                       // token row of S; dim (mod 128) of O^T
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t spread = spread_of(row);
    auto sync_all = [] { asm volatile("bar.sync 7, %0;" ::"n"(kWarps * 32) : "memory"); };        // the softmax warps
    auto sync_group = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); };     // the group's four
    Ring s_ring, sc_ring;
    int it = 0;
#pragma unroll 1
    for (int u = u_begin; u < u_end;) {
      const Piece pc = piece_at(u);
      u += pc.span;
      const int q0 = bd.q_indptr[pc.b], n_nodes = bd.q_indptr[pc.b + 1] - q0;
      const int hpc = min(p.hpc, p.group - pc.c * p.hpc);
      const int head0 = pc.g * p.group + pc.c * p.hpc;
      const int rows = hpc * n_nodes, nc = (rows + 15) / 16;
      // 16-column chunks of this group.  It always computes CC of them (straight code); what lies past the columns in use
      // is never multiplied, and its references below every score keep it out of the way.
      const int mine = min(CC, max(0, nc - group * CC)), c_first = group * CC;
      const int col0 = c_first * 16;
      const bool has_draft = pc.first == 0;
      // ---------------------------------------------------------- staging: Q, the tree, the draft block
      // (the previous piece's products have all finished: its last O_DONE was waited for)
      if (tid < n_nodes) {
        const int up = p.parents[q0 + tid];
        sm->par[tid] = (int8_t)(up < -1 || up >= kMaxNodes ? -2 : up);
      }
      {
        // Rows by warp; a warp's query rows all at once, then, in the draft CTA, the block's K and V rows.  The code runs
        // once per piece: it is kept short, since its first run waits for its own instructions.
        constexpr int LPR = D / 8, RPW = 32 / LPR;                     // lanes per row, rows per warp and load
        constexpr int U = (NQ + kWarps * RPW - 1) / (kWarps * RPW);    // a warp's query rows, RPW at a time
        const int sub = lane / LPR, ch = lane % LPR;                   // 8-value chunk of the row
        const int n_q = nc * 16;
        const float inv_hpc = 1.0f / (float)hpc;
        auto row_amax = [&](uint4& x, bool& wild) {        // a row with a NaN or an infinity counts as zeros
          uint32_t a = amax_bits(x);
          if (RPW == 1) {
            a = __reduce_max_sync(0xffffffffu, a);
          } else {
#pragma unroll
            for (int d = LPR / 2; d >= 1; d >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
          }
          wild = a >= 0x7f80u;
          if (wild) x = make_uint4(0, 0, 0, 0);
          return wild ? 0u : a;
        };
        const uint32_t ch_off = (uint32_t)((ch & 1) << 3), ch_chunk = (uint32_t)(ch >> 1) & 7u;
        auto swizzled = [&](int r) { return (((ch_chunk ^ (uint32_t)r) & 7u) << 4) + ch_off; };
        uint4 x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int r = (i * kWarps + warp) * RPW + sub;
          const int node = __float2int_rz(((float)r + 0.5f) * inv_hpc);   // r / hpc, exact for r < 2^20
          x[i] = make_uint4(0, 0, 0, 0);
          if (r < rows)
            x[i] = __ldg(reinterpret_cast<const uint4*>(p.q + (long long)(q0 + node) * p.q_stride +
                                                        (head0 + r - node * hpc) * D) + ch);
        }
        if (has_draft) {
          // the ring slots of the draft tile, once their previous contents have been multiplied
          spin(B_KE + it % KS, it / KS + 1);
          spin(B_VE + 2 * it % VS, 2 * it / VS + 1);
          spin(B_VE + (2 * it + 1) % VS, (2 * it + 1) / VS + 1);
          uint8_t* const k_hi = sK + it % KS * K::kTileBytes;
          uint8_t* const v_hi = sV + 2 * it % VS * K::kHalf;
          uint8_t* const v_lo = sV + (2 * it + 1) % VS * K::kHalf;
          // rows 0 .. n - 1: K, n .. 2 n - 1: V; then zeros up to V's 32-token step
          const int v_end = n_nodes + ((n_nodes + 31) & ~31);
#pragma unroll 1
          for (int base = warp * RPW; base < v_end; base += kWarps * RPW) {
            const int r = base + sub;
            const bool is_v = r >= n_nodes;
            const int n = is_v ? r - n_nodes : r;
            uint4 y = make_uint4(0, 0, 0, 0);
            if (n < n_nodes)
              y = __ldg(reinterpret_cast<const uint4*>((is_v ? p.v_new + (long long)(q0 + n) * p.v_stride
                                                             : p.k_new + (long long)(q0 + n) * p.k_stride) + pc.g * D) + ch);
            bool wild = false;
            int e = 0;
            uint2 hi = make_uint2(0, 0), lo = hi;
            if (base < 2 * n_nodes) {      // zero rows are stored as they are (512-token decode 11.6 -> 10.9 us)
              e = exp_of(row_amax(y, wild));
              split8(y, exp2i(-e), hi, lo);
            }
            if (r < v_end) {
              const uint32_t off = (uint32_t)((n >> 3) * K::kGroupBytes + (ch >> 4) * 1024 + (n & 7) * 128) + swizzled(n);
              *reinterpret_cast<uint2*>((is_v ? v_hi : k_hi) + off) = hi;
              *reinterpret_cast<uint2*>((is_v ? v_lo : k_hi + 8 * K::kGroupBytes) + off) = lo;
              if (ch == 0 && n < n_nodes) (is_v ? sm->row_v : sm->row_k)[n] = wild ? __int_as_float(0x7fc00000) : exp2i(e);
            }
          }
        }
        int e_q[U];
        uint32_t wilds = 0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          bool wild;
          e_q[i] = query_exp(row_amax(x[i], wild));
          wilds |= wild ? 1u << i : 0u;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int r = (i * kWarps + warp) * RPW + sub;
          uint2 hi, lo;
          split8(x[i], exp2i(-e_q[i]), hi, lo);
          if ((wilds >> i) & 1u) hi = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);     // NaN codes: the column's scores are NaN
          if (r < n_q) {
            uint8_t* at = sQ + (ch >> 4) * NQ * 128 + r * 128 + swizzled(r);
            *reinterpret_cast<uint2*>(at) = hi;
            *reinterpret_cast<uint2*>(at + K::kQTerm) = lo;
            if (ch == 0) sm->qf[r] = exp2i(e_q[i]);
          }
        }
      }
      fence_async_smem();
      sync_all();
#pragma unroll 1
      for (int q = tid; q < NQ; q += kWarps * 32) {
        sm->m[q] = q < nc * 16 ? 0.f : -1e30f;     // no reference yet; columns past those in use: below everything
        if (q >= nc * 16) sm->qf[q] = 1.f;
        if (MOD) sm->slope[q] = p.slopes != nullptr && q < rows ? p.slopes[head0 + q % hpc] * kLog2e : 0.f;
      }
      // the tree: root paths and depths
      if (tid < n_nodes) {
        unsigned long long a = 1ull << tid;
        int d = 0;
        bool good = sm->par[tid] >= -1 && (tid > 0 || sm->par[0] == -1);
#pragma unroll 1
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
      sync_all();
      if (tid == 0) mbar_arrive(bar(B_Q));
      if (has_draft && n_nodes > 1) {
        // While the first product runs: the root paths turned round by ballots, a row of the tile a turn.  (Asked node by
        // node in the tile they took 90 ns a node: 89 sequences of up to 62 nodes 475 -> 423 us.)
        unsigned long long a0 = 0, a1 = 0;
        int d0 = 0, d1 = 0;
        if (lane < n_nodes) { a0 = sm->anc[lane]; d0 = sm->depth[lane]; }
        if (lane + 32 < n_nodes) { a1 = sm->anc[lane + 32]; d1 = sm->depth[lane + 32]; }
        sync_all();
#pragma unroll 1
        for (int r = warp; r < n_nodes; r += kWarps) {
          const int far = p.window > 0 && p.window < kMaxNodes ? sm->depth[r] + p.window : INT_MAX;   // the depth that no longer sees it
          const uint32_t lo = __ballot_sync(0xffffffffu, ((a0 >> r) & 1ull) != 0ull && d0 < far);
          const uint32_t hi = __ballot_sync(0xffffffffu, ((a1 >> r) & 1ull) != 0ull && d1 < far);
          if (lane == 0) sm->anc[r] = (unsigned long long)hi << 32 | lo;
        }
        sync_all();
      }

      float2 sum[CC][8];
#pragma unroll
      for (int c = 0; c < CC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[c][e] = make_float2(0.f, 0.f);
      const int lo_root = p.window > 0 ? pc.L - p.window + 1 : 0;
      // The scales of this thread's token row in the coming tile: the score factor, log2 of the V scale, and the V scale
      // on the weights.
      const float fac = p.scale * kLog2e;
      float kf, lv, vd;
      auto set_scales = [&](float ks, float vs) {
        kf = ks * fac;
        lv = fast_log2(vs);
        vd = vs * kDown;
      };
      auto next_scales = [&] {
        set_scales(sm->scale[sc_ring.at][row >> 4], sm->scale[sc_ring.at][8 + (row >> 4)]);
        sc_ring.next(SC);
      };
      if (has_draft) {
        const float rv = row < n_nodes ? sm->row_v[row] : 1.f;
        set_scales(row < n_nodes ? sm->row_k[row] : 1.f, rv != rv ? 1.f : rv);
        sc_ring.next(SC);
      } else {
        wait_full(B_SC, sc_ring);
        __syncwarp();
        next_scales();
      }

      // The scores of this token row, drawn at the end of the turn before; S is then free for the tile after the next.
      float a[CC][16];
      auto draw = [&] {
        __syncwarp();
        tc_fence_after();
        const uint32_t s_addr = tmem + lane_addr + s_ring.at * NQ + col0;
#pragma unroll
        for (int c = 0; c < CC; ++c) tmem_ld16(s_addr + c * 16, a[c]);
        tmem_wait_ld();
      };
      auto drawn = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_SE + s_ring.at));
        s_ring.next(NS);
      };
      wait_full(B_SF, s_ring);
      draw();
      drawn();
      // Until a tile that every column sees something of has passed, columns may have no reference.
      bool settled = false;
#pragma unroll 1
      for (int i = 0; i < pc.tiles; ++i, ++it) {
        const bool draft = pc.first + i == 0;
        const int t0 = pc.t0(pc.first + i);
        const int valid = draft ? n_nodes : min(kTile, pc.L - t0);
        const bool band = !draft && p.window > 0 && t0 < lo_root + kMaxNodes;
        const bool masked = draft || valid < kTile || band;
        if (band && t0 + row >= lo_root && t0 + row < min(pc.L, lo_root + kMaxNodes)) {
          // a token that a window may hide from some nodes: its NaN codes of V become NaN scores
          const int pg = p.page_table[(size_t)pc.b * p.max_pages + (t0 + row) / kPage];
          if (pg >= 0 && pg < p.num_pool_pages) {
            const uint4* src = reinterpret_cast<const uint4*>(
                p.v_cache + (((size_t)pg * p.hkv + pc.g) * kPage + (t0 + row) % kPage) * D);
            uint32_t nan = 0;
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) {
              const uint4 v = __ldg(src + e);
              nan |= __vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                     __vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
            }
            if (nan != 0u) kf = __int_as_float(0x7fc00000);
          }
        }
        // ---- exponents against the references as they stand (base 2), and the chunks where a weight would pass kTop
        uint32_t missed = 0;
        const float limit = 8.807354922f - lv;       // log2(kTop)
        // the bias' distance is counted from the root: a node's depth shifts all its scores alike (see the log-sum-exp)
        const float rel = draft ? (row < n_nodes ? (float)sm->depth[row] : 0.f) : (float)(t0 + row - pc.L);
        // A product becomes a score by its token's factor, then its column's (in this order nothing overflows that the
        // score itself does not).
        auto scored = [](float x, float y, float token, float qx, float qy) {
          return mul2(mul2(make_float2(x, y), make_float2(token, token)), make_float2(qx, qy));
        };
        float kv = kf;
        const bool cap = MOD && p.softcap > 0.f;
        if (cap) {
          // c tanh(x / c) = c - 2 c / (1 + 2^(2 log2e x / c)): off by some c 2^-22, 1e-5 nats at the 30 to 50 of models with
          // capped scores and 1e-3 at the largest cap that a call takes.  (A second form without the difference for large
          // caps, tanh's Taylor series near 0, costs the others 1.7 us of 42 by its branch alone: the tree of 31.)
          const float cl = p.softcap * kLog2e, ky = kf * p.cap_exp;
#pragma unroll
          for (int c = 0; c < CC; ++c) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 qf = *reinterpret_cast<const float2*>(&sm->qf[col0 + c * 16 + e]);
              const float2 y = scored(a[c][e], a[c][e + 1], ky, qf.x, qf.y);
              const float2 d = add2(make_float2(fast_exp2(y.x), fast_exp2(y.y)), make_float2(1.f, 1.f));
              const float2 s = fma2(make_float2(fast_rcp(d.x), fast_rcp(d.y)), make_float2(-2.f * cl, -2.f * cl), make_float2(cl, cl));
              a[c][e] = s.x;
              a[c][e + 1] = s.y;
            }
          }
          kv = 1.f;
        }
#pragma unroll
        for (int c = 0; c < CC; ++c) {
          const int q = col0 + c * 16;
          float top = -INFINITY;      // of this chunk
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 m = *reinterpret_cast<const float4*>(&sm->m[q + 4 * k]);
            float* v = &a[c][4 * k];
            float2 m0 = make_float2(m.x, m.y), m1 = make_float2(m.z, m.w);
            if (MOD) {
              const float4 sl = *reinterpret_cast<const float4*>(&sm->slope[q + 4 * k]);
              m0 = fma2(make_float2(sl.x, sl.y), make_float2(rel, rel), m0);
              m1 = fma2(make_float2(sl.z, sl.w), make_float2(rel, rel), m1);
            }
            const float4 qf = *reinterpret_cast<const float4*>(cap ? sm->one : &sm->qf[q + 4 * k]);
            const float2 d0 = fma2(mul2(make_float2(v[0], v[1]), make_float2(kv, kv)), make_float2(qf.x, qf.y), m0);
            const float2 d1 = fma2(mul2(make_float2(v[2], v[3]), make_float2(kv, kv)), make_float2(qf.z, qf.w), m1);
            v[0] = d0.x; v[1] = d0.y; v[2] = d1.x; v[3] = d1.y;
            top = fmaxf(fmaxf(top, fmaxf(d0.x, d0.y)), fmaxf(d1.x, d1.y));
          }
          missed |= top > limit ? 1u << c : 0u;
        }
        if (__any_sync(0xffffffffu, missed != 0u)) missed = __reduce_or_sync(0xffffffffu, missed);
        const uint32_t all = (1u << mine) - 1u;
        missed &= all;
        if (masked) {
          // Which columns see this row: one bit each.  Masked exponents are -inf whatever the product was.
          using Bits = typename BitsOf<CC>::type;
          Bits vis = row < valid && !draft && !band ? ~(Bits)0 : 0;
          if (row < valid && (draft || band)) {
            // node by node, from the one of the group's first column: its columns see this row, or none of them does
            int n = col0 / hpc, at = n * hpc - col0;       // the node's first column, less the group's
            const Bits full = ((Bits)1 << hpc) - 1;
            Bits bits = full >> -at;
            if (draft) {
              unsigned long long seen = n < n_nodes ? sm->anc[row] >> n : 0ull;
#pragma unroll 1
              for (; at < CC * 16 && seen != 0ull; seen >>= 1) {
                vis |= seen & 1ull ? bits : (Bits)0;
                at += hpc;
                bits = full << (at & (8 * (int)sizeof(Bits) - 1));
              }
            } else {
#pragma unroll 1
              for (; at < CC * 16 && n < n_nodes; ++n) {
                vis |= t0 + row >= lo_root + sm->depth[n] ? bits : (Bits)0;
                at += hpc;
                bits = full << (at & (8 * (int)sizeof(Bits) - 1));
              }
            }
          }
#pragma unroll
          for (int c = 0; c < CC; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) a[c][e] = ((uint32_t)(vis >> (CC > 2 ? c / 2 * 32 : 0)) >> ((c & 1) * 16 + e)) & 1u ? a[c][e] : -INFINITY;
        }
        // ---- the weights, on the assumption that no warp of the group has to move a reference; what they need to know
        // of each other is under way meanwhile.  (The barrier also keeps red[] of this tile behind the last one's readers.)
        uint32_t hi[CC][4], lo[CC][4];
        auto weigh = [&](int c, float add) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 e0 = make_float2(fast_exp2(a[c][4 * k]), fast_exp2(a[c][4 * k + 1]));
            const float2 e1 = make_float2(fast_exp2(a[c][4 * k + 2]), fast_exp2(a[c][4 * k + 3]));
            sum[c][2 * k] = fma2(e0, make_float2(add, add), sum[c][2 * k]);
            sum[c][2 * k + 1] = fma2(e1, make_float2(add, add), sum[c][2 * k + 1]);
            split4(mul2(e0, make_float2(vd, vd)), mul2(e1, make_float2(vd, vd)), spread, hi[c][k], lo[c][k]);
          }
        };
        const bool plain = settled && !masked;
        if (!plain) missed = all;
        if (lane == 0) {
          sm->flag[group][it & 1][quarter] = (int)missed;
          mbar_arrive(bar(B_G + group));
        }
        if (plain) {
          if (MOD && missed == 0u) {
#pragma unroll
            for (int c = 0; c < CC; ++c) weigh(c, 1.f);
          } else {
#pragma unroll
            for (int c = 0; c < CC; ++c)
              if (!((missed >> c) & 1u)) weigh(c, 1.f);
          }
        }
        settled = settled || draft || !band;
        spin(B_G + group, it);
        const int4 fl = *reinterpret_cast<const int4*>(sm->flag[group][it & 1]);
        const uint32_t todo = (uint32_t)(fl.x | fl.y | fl.z | fl.w);     // chunks whose references move
        if (todo != 0u) {
          // The exact maxima of these chunks' columns, new references (unset ones are 0, set ones never are),
          // and the weights and sums against them.
#pragma unroll
          for (int c = 0; c < CC; ++c) {
            if ((todo >> c) & 1u) {
              const float mx = warp_max16(a[c], lv, lane);
              if (lane < 16) sm->red[quarter][col0 + c * 16 + lane] = mx;
            }
          }
          sync_group();
          const int mine_col = quarter * 32 + lane, q = col0 + mine_col;
          if (mine_col < mine * 16 && ((todo >> (mine_col >> 4)) & 1u)) {
            const float old = -sm->m[q];
            const float mt = old + fmaxf(fmaxf(sm->red[0][q], sm->red[1][q]), fmaxf(sm->red[2][q], sm->red[3][q])) -
                             head_of(pc.tiles, old == 0.f);
            float now = mt == -INFINITY ? old : old == 0.f ? mt : fmaxf(old, mt);
            if (now == 0.f && mt != -INFINITY) now = 1e-30f;
            sm->alpha[q] = old == 0.f ? 1.f : fast_exp2(old - now);
            sm->m[q] = -now;
            sm->red[0][q] = old - now;
          }
          sync_group();
#pragma unroll
          for (int c = 0; c < CC; ++c) {
            if ((todo >> c) & 1u) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 al = *reinterpret_cast<const float2*>(&sm->alpha[col0 + c * 16 + 2 * e]);
                const float2 dl = *reinterpret_cast<const float2*>(&sm->red[0][col0 + c * 16 + 2 * e]);
                sum[c][e] = mul2(sum[c][e], al);
                a[c][2 * e] += dl.x;
                a[c][2 * e + 1] += dl.y;
              }
              weigh(c, (missed >> c) & 1u ? 1.f : 0.f);     // 0: this tile's weights are in the sum
            }
          }
        }
        // the coming tile's scales while the previous tile's PV runs, if they are there
        const bool last = i + 1 >= pc.tiles;
        bool ahead = last;
        if (NG > 1 && !ahead) {
          ahead = __all_sync(0xffffffffu, mbar_test(bar(B_SC + sc_ring.at), sc_ring.round));
          if (ahead) next_scales();
        }
        // P and O belong to the previous tile's PV until it has finished
        if (it > 0) spin(B_OD, it - 1);
        tc_fence_after();
        if (todo != 0u && i > 0) {
#pragma unroll 1
          for (int c = 0; c < mine; ++c) {
            if (!((todo >> c) & 1u)) continue;
#pragma unroll 1
            for (int mb = 0; mb < MH; ++mb) {
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
        for (int c = 0; c < CC; ++c) {
          uint8_t* at = sP + (c_first + c) * kTile * 16 + row * 16;
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[c][0], hi[c][1], hi[c][2], hi[c][3]);
          *reinterpret_cast<uint4*>(at + K::kPTerm) = make_uint4(lo[c][0], lo[c][1], lo[c][2], lo[c][3]);
        }
        tc_fence_before();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PF));
        if (!ahead) {
          wait_full(B_SC, sc_ring);
          __syncwarp();
          next_scales();
        }
        // (Past the last tile S holds old scores, which nobody uses: drawn all the same, a condition here costs the wide
        // tiles registers that they do not have, and 89 us become 91.)
        if (!last) wait_full(B_SF, s_ring);
        draw();
        if (!last) drawn();
      }

      // ---------------------------------------------------------- results
      // Column sums over the tile's 128 token rows: the lanes, then the quarters.
      sync_group();      // the last tile's readers of red[] are done
#pragma unroll
      for (int c = 0; c < CC; ++c) {
        {
          float v[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) { v[2 * e] = sum[c][e].x; v[2 * e + 1] = sum[c][e].y; }
          const float s = warp_sum16(v, lane);
          if (lane < 16) sm->red[quarter][col0 + c * 16 + lane] = s;
        }
      }
      sync_group();
      spin(B_OD, it - 1);
      tc_fence_after();
      const size_t slot = (size_t)blockIdx.x + pc.seg;      // rises by at least one along the pieces: unique
      {
        const int q = col0 + quarter * 32 + lane;
        if (quarter * 32 + lane < mine * 16) {
          const float l = sm->red[0][q] + sm->red[1][q] + sm->red[2][q] + sm->red[3][q];
          sm->alpha[q] = l == 0.f ? 0.f : 1.f / l;
          // the column's output row, in place of its sums
          int* out_row = reinterpret_cast<int*>(sm->red[0]);
          out_row[q] = -1;
          if (q < rows) {
            const int node = q / hpc, at = (q0 + node) * p.hq + head0 + q - node * hpc;
            out_row[q] = pc.whole ? at : q;
            float lse2 = l == 0.f ? -INFINITY : fast_log2(l) - sm->m[q];
            if (MOD) lse2 -= sm->slope[q] * (float)sm->depth[node];
            if (!pc.whole) p.lse_part[slot * NQ + q] = lse2;
            else if (p.lse != nullptr) p.lse[at] = lse2 * kLn2;
          }
        }
      }
      sync_group();
#pragma unroll 1
      for (int c = 0; c < mine; ++c) {
        float v[MH][16];
#pragma unroll
        for (int mb = 0; mb < MH; ++mb) tmem_ld16(tmem + lane_addr + kColO + mb * NQ + col0 + c * 16, v[mb]);
        tmem_wait_ld();
        const float* inv = sm->alpha + col0 + c * 16;
        const int* at = reinterpret_cast<const int*>(sm->red[0]) + col0 + c * 16;
        if (pc.whole) {
          const bool odd = lane & 1;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = at[2 * k + odd];
#pragma unroll
            for (int mb = 0; mb < MH; ++mb) {
              const float ev = v[mb][2 * k] * inv[2 * k], od = v[mb][2 * k + 1] * inv[2 * k + 1];
              // even lanes keep the even column and take the odd lane's dim of it; odd lanes the reverse
              const float got = __shfl_xor_sync(0xffffffffu, odd ? ev : od, 1);
              const __nv_bfloat162 h = __floats2bfloat162_rn(odd ? got : ev, odd ? od : got);
              if (r >= 0) *reinterpret_cast<__nv_bfloat162*>(p.out + (size_t)r * D + mb * 128 + (row & ~1)) = h;
            }
          }
        } else {
          // the columns' rows follow each other in the partial
          float* dst = p.o_part + (slot * NQ + col0 + c * 16) * D + row;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
#pragma unroll
            for (int mb = 0; mb < MH; ++mb)
              if (col0 + c * 16 + k < rows) dst[k * D + mb * 128] = v[mb][k] * inv[k];
          }
        }
      }
      tc_fence_before();
      // every warp is done with the columns' arrays and O before the next piece is staged
      sync_all();
      tc_fence_after();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm->abort) report(p.dev_status, SD_DEV_TIMEOUT);
  if (warp == kWarpQK) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(K::kTmem));
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace
}  // namespace sdv
