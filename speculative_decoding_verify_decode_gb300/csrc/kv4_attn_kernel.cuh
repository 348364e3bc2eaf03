// Verify attention over the 4-bit cache (include/sd_kv4.h: sd_kv4_attn):
// codes widened in registers into tensor memory, tcgen05 products from there.
//
// The mathematics.  A query column is one (draft node, query head) pair of a
// KV head; a key is a context token with k, v = (c - 8) s, or a draft node.  With
// s = cap(scale q.k) + bias in base 2 and a running reference m of the column,
//   e = 2^(s - m),   l += e,   O += bf16(e) v,   out = O / l.
// (c - 8) s is exactly a bf16 value, so the products are those of a bf16 cache
// that holds what the codes stand for.  m is the first tile's maximum, and moves
// (with O and l rescaled) only when a weight passes 2^kRise: fp32 sums and bf16
// weights are as exact at 2^16 as at 1.  Weights are bf16 because both operands of
// a kind::f16 product have one type, and V's values need bf16's exponents: outputs
// are off by 0.0018 to 0.0023 of their size, 0.0017 of it the output's own rounding.
//
// Where the widened operand goes.  A tile's 128 tokens x D dims (or D dims x 128
// tokens of V^T) are the MMA's A operand, which may lie in tensor memory with a row
// per lane: a thread takes its row's codes out of shared memory (16 bytes are 32
// values), makes pairs of bf16 with three instructions each, and stores them to its own lane.
// Nothing widened passes through shared memory, where the same tile would be
// written and read at four times its size.  The cache's records are laid out for it: K's
// words go along a token's dims, V's along a dim's tokens, so neither is transposed.
//
// What bounds it.  Bytes: 9 D / 16 a token and KV head for K and as many for V, read once per CTA column part: 1570 cycles
// a tile of 256 dims at an SM's share of HBM.  Single tokens (16 columns): the instructions of the widening, some 1000
// a tile and scheduler, half of them integer ones of two cycles (64 sequences of 1 to 32768 tokens, 128 dims: 382 us where
// the bytes take 207; of 1 to 16384, 256 dims: 188 of 104).  144 columns of 256 dims: 32 products of 81 cycles, then the chain
// S -> softmax -> S, as there is one S buffer and 1152 cycles of exponentials (a tile takes 4700 cycles; a tree of 23 over
// 131072 tokens 89.5 us, where its operations take 38 and its bytes 22).  Between them, 96 columns: 3300 cycles a tile.  A piece costs as much as three to five tiles
// more: query rows and the tree are staged, the first references are taken, partial outputs are stored.
//
// Work split, line of units, pieces and merge: as in kv8_attn_kernel.cuh.
//
// Per tile (tokens are the MMA's M; NQ columns):
//   S[128 tok][NQ]     = K_tile . Q^T          A from tensor memory, Q K-major in shared memory
//   O^T[D][NQ]        += V_tile^T . P^T        M = 128 dims a product, P MN-major in shared memory
// Warps: NG groups of four softmax warps (lane quarter = warp % 4, CC chunks of 16 columns a
// group; thread = token row), WG groups of KG x 4 that widen K and of four that widen V, then one each that loads K,
// loads V, issues QK, issues PV.  The softmax reads its scores once: it forms weights with the references that there are,
// and where one is beyond 2^kRise, or there is none yet, the group moves these columns' references and forms them anew.
// Masked, capped or biased scores are formed first and go back to S.
// Every wait on a barrier is bounded; on expiry the kernel reports
// SD_DEV_TIMEOUT and runs out.
#pragma once

#include <cstddef>

#include "kernels.h"
#include "kv4_format.cuh"
#include "tc_ptx.cuh"

namespace sdv {
namespace {

constexpr int kTile = kTileTokens;     // tokens of a product's M
constexpr float kRise = 16.0f;         // log2 of the weight beyond which a reference moves
constexpr float kLarge = 67108864.0f;  // 2^26: a reference beyond which scores are rounded before it is taken off (see `large`)
constexpr float kLog2e = 1.4426950408889634f;

template <int NQ, int VW, int MH, bool MOD>
struct Kv4Small {
  static constexpr int kBars = 56;
  float m[NQ];             // the column's reference, negated: -m
  float alpha[NQ];         // rescale factor of the current tile; 1 / l in the epilogue
  float slope[MOD ? NQ : 4];   // distance bias of the column, base 2
  float red[4][NQ];        // per lane quarter: column maxima of a tile; column sums in the epilogue
  alignas(16) uint2 vs[VW][MH][64];           // per V warp: scales of a tile's token pairs, and -24 times them
  unsigned long long anc[kMaxNodes];          // bit r: node r is on the node's root path; in the draft CTA then turned
                                              // round, bit n: node n sees the row
  uint64_t bar[kBars];
  int cum[kMaxBatch + 1];  // first unit of each sequence
  int scan[8];
  int per, extra;
  int8_t par[kMaxNodes];
  int8_t depth[kMaxNodes];
  int8_t wild[kMaxNodes];  // the node's key or value holds a NaN or an infinity
  alignas(16) int flag[3][2][4];   // [group][tile parity][lane quarter]: chunks where a weight passes 2^kRise
  int large[3];                    // [group]
  uint32_t tmem;
  int abort;
};

// D: head dim.  NG groups of softmax warps, of up to CC 16-column chunks each.  MOD: capped scores or a distance bias.
template <int D, int NG, int CC, bool MOD>
struct Kv4 {
  static constexpr int NQ = NG * CC * 16;                 // query columns
  // Groups of four warps that widen K, and as many that widen V, tile by tile in turn; each has rings of its own (what is
  // counted below), so that no barrier has a user that passes some of its phases by.
  // Single tokens: half a CTA's columns, and where a tile is large (256 dims) two CTAs, of which one works while the other
  // goes from piece to piece (64 sequences of 1 to 16384 tokens 236 -> 213 us, one of 512 tokens 12.4 -> 11.4); of 128
  // dims one CTA with two groups is faster (64 sequences of 1 to 32768 tokens 427 us against 463).
  static constexpr int kCtas = kv4_ctas(NQ, D);
  static constexpr int WG = NQ == 16 && kCtas == 1 ? 2 : 1;
  // 144 columns: tensor memory has room for short slots only, and one S buffer, so the widening of K is waited for.  Each of
  // its two slots has a group of four warps of its own, which widens its next values before the slot is free, and the
  // products of QK go before those of PV (tree of 23 over 131072 tokens 97 -> 91 us; the other widths gain nothing by it).
  static constexpr int KG = NQ < 144 ? 1 : 2;
  static constexpr int kWarps = NG * 4, kWideK = WG * KG * 4, kWideV = WG * 4, kThreads = (kWarps + kWideK + kWideV + 4) * 32;
  // Registers of the launch, and the roles' shares of them.
  static constexpr int kLaunchRegs = 65536 / kCtas / kThreads / 8 * 8;
  static constexpr int kRegsSoft = kCtas == 2 ? 88 : NG == 3 ? 104 : 136;
  static constexpr int kRegsWide = kCtas == 2 ? 64 : NG == 3 ? 48 : 72;
  static constexpr int kRegsRest = kCtas == 2 ? 40 : NG == 3 ? 40 : 56;
  static_assert(kWarps * kRegsSoft + (kWideK + kWideV) * kRegsWide + 4 * kRegsRest <= kThreads / 32 * kLaunchRegs, "registers");
  static constexpr int kSmemBytes = kCtas == 2 ? 115712 : 232448;   // dynamic shared memory a CTA can have
  static constexpr int kTmem = 512 / kCtas;
  static constexpr int MH = D / 128;                      // 128-dim blocks
  using Small = Kv4Small<NQ, kWideV, MH, MOD>;
  // Tiles that pass the softmax together: what a turn costs beyond them (barriers, the references' check, bookkeeping)
  // is as much as sixteen columns of a tile or two (64 sequences, 128 dims: one tile 560 us, four 427).
  static constexpr int T = NQ == 16 && kCtas == 1 ? 4 : NQ <= 48 ? 2 : 1;
  static constexpr int NS = NQ <= 96 || D == 128 ? 2 : 1; // S buffers in tensor memory
  // Widened operands: slots of SW elements a lane, two to a column.  One long slot beats two short ones, whose handshakes
  // cost more than their overlap gives (8 chains of 5 nodes: 64 elements 39 us, 128 36); 144 columns leave no room for it.
  static constexpr int SW = NQ < 144 ? 128 : 32;
  static constexpr int kSlotCols = SW / 2;
  // Short slots: the first values are widened before their slot is waited for.
  static constexpr bool kEarly = SW < 128;
  static constexpr int kColO = NS * T * NQ, kColA = kColO + MH * NQ;
  static constexpr int kSlotsLeft = (kTmem - kColA) / kSlotCols / WG;
  static constexpr int KA = kSlotsLeft / 2 > 1 && D / SW > 1 ? 2 : 1, VA = kSlotsLeft - KA > 1 && kTile / SW * MH > 1 ? 2 : 1;
  // A tile takes the ring round KU (VU) times: which slot, and which phase of it, is known without counting.
  static constexpr int KU = D / SW / KA, VU = kTile / SW * MH / VA;
  static constexpr int kRecord = kv4_record(D), kTileBytes = 8 * kRecord;   // a page's K or V; a tile's
  static constexpr int kQBytes = NQ * D * 2;
  static constexpr int kPBytes = NQ * T * kTile * 2;      // [8-column chunk][token][16 bytes]
  static constexpr int kLeft = (kSmemBytes - kQBytes - 2 * kPBytes - (int)sizeof(Small)) / kTileBytes;
  // A page's K and V lie together: one ring of both where it holds eight tiles, else a ring each (V is needed later than K).
  static constexpr bool kJoint = kLeft >= 16;
  static constexpr int kUnits = kLeft > 20 ? 20 : kLeft;
  static constexpr int KS = kUnits / 2 / WG, VS = kJoint ? KS : kUnits / WG - KS;
  static constexpr int kPageStride = kJoint ? 2 * kRecord : kRecord, kSlotBytes = 8 * kPageStride;
  static constexpr size_t kRingBytes = (size_t)(kJoint ? KS : KS + VS) * WG * kSlotBytes;
  static constexpr size_t kSmem = (size_t)kQBytes + 2 * kPBytes + kRingBytes + sizeof(Small);
  static_assert(KG == 1 || KA == KG, "a slot for each group");
  static_assert(KS * WG >= 2 && VS * WG >= 2, "rings of two tiles at least");
  static_assert(kColA + WG * (KA + VA) * kSlotCols <= kTmem, "tensor memory");
  static_assert(KU * KA * SW == D && VU * VA * SW == kTile * MH, "slots of a tile");
  static_assert(kSmem <= (size_t)kSmemBytes, "shared memory over 227 KB");
};

// ------------------------------------------------------------ small pieces

// A bounded wait: false, with the CTA's abort flag set, if the phase never completes.  The kernel's end reports the flag.
__device__ __forceinline__ bool wait4(uint32_t bar, uint32_t parity, volatile int* abort) {
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
// One lane of a converged warp (the tensor core's and TMA's instructions take uniform operands).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ uint64_t noswz_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}
// kind::f16, A in tensor memory (128 lanes, two K elements a column), B in shared memory.
// ACC: 1 adds to D, 2 as `acc` says.
template <int ACC>
__device__ __forceinline__ void umma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc = 1) {
  if (ACC == 2)
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc));
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "n"(ACC));
}
// A record of one page (a multiple of 16 bytes), read with the evict-first policy.
__device__ __forceinline__ void bulk_record(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
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
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tcgen05.wait::ld, with the values that it was waited for (whose uses then cannot come before it).
__device__ __forceinline__ void wait_scores(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
// Maxima of 16 values over the warp's lanes: lane L ends with that of value L % 16.
__device__ __forceinline__ float warp_max16(const float (&v)[16], int lane) {
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(x) : "f"(v[i]));
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
__device__ __forceinline__ bool wild8(const uint4 x) {   // a NaN or an infinity among eight bf16 values
  const uint32_t e = 0x7f807f80u;
  return (__vcmpeq2(x.x & e, e) | __vcmpeq2(x.y & e, e) | __vcmpeq2(x.z & e, e) | __vcmpeq2(x.w & e, e)) != 0u;
}

// What a segment's draft tile counts for beyond one unit, where CTAs have `even` units each: staging and the first
// references take as long as a few tiles; in pieces of few units one more would cost the whole.
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
__global__ void __launch_bounds__(Kv4<D, NG, CC, MOD>::kThreads, Kv4<D, NG, CC, MOD>::kCtas)
kv4_attn_kernel(const Kv4AttnParams p, const BatchDesc bd) {
  using K = Kv4<D, NG, CC, MOD>;
  constexpr int NQ = K::NQ, MH = K::MH, NS = K::NS, KS = K::KS, VS = K::VS, KA = K::KA, VA = K::VA, SW = K::SW, WG = K::WG, KG = K::KG,
                T = K::T;
  constexpr int kWarps = K::kWarps, kAllThreads = K::kThreads;      // softmax warps; all threads
  constexpr int kWarpWideK = kWarps, kWarpWideV = kWarps + K::kWideK, kWarpK = kWarpWideV + K::kWideV, kWarpV = kWarpK + 1,
                kWarpQK = kWarpK + 2;
  using Sm = typename K::Small;
  constexpr int B_KF = 0, B_KE = B_KF + KS * WG, B_VF = K::kJoint ? B_KF : B_KE + KS * WG, B_VE = K::kJoint ? B_KE : B_VF + VS * WG,
                B_AKF = B_VE + VS * WG, B_AKE = B_AKF + KA * WG, B_AVF = B_AKE + KA * WG, B_AVE = B_AVF + VA * WG, B_SF = B_AVE + VA * WG, B_SE = B_SF + 2, B_PF = B_SE + NS,
                B_OD = B_PF + 2, B_Q = B_OD + 2, B_G = B_Q + 1;
  constexpr int kNumBars = B_G + NG;
  static_assert(kNumBars <= Sm::kBars, "barriers");
  extern __shared__ __align__(1024) uint8_t smem4[];
  uint8_t* sQ = smem4;
  uint8_t* sP = sQ + K::kQBytes;                 // two buffers
  uint8_t* sK = sP + 2 * K::kPBytes;
  uint8_t* sV = K::kJoint ? sK + K::kRecord : sK + KS * WG * K::kSlotBytes;
  Sm* sm = reinterpret_cast<Sm*>(sK + K::kRingBytes);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (smem_u32(smem4) & 1023u) {   // not expected; refuse rather than mis-swizzle
    if (tid == 0) report_dep(p.dev_status, SD_DEV_TIMEOUT);
    return;
  }

  // ---------------------------------------------------------------- the line of units
  const int parts = p.hkv * p.hparts;   // segments per sequence
  auto ctx_of = [&](int b) {
    const int L = p.ctx_lens[b];
    return L < 0 ? 0 : min(L, p.max_pages * kPage);
  };
  if (tid < kNumBars) {
    const int i = tid;
    const bool k_empty = i >= B_KE && i < B_KE + KS * WG, v_empty = i >= B_VE && i < B_VE + VS * WG;     // both where the ring is joint
    const bool by_four = (i >= B_AKF && i < B_AKE) || (i >= B_AVF && i < B_AVE) || i >= B_G;
    const bool by_softmax = (i >= B_SE && i < B_SE + NS) || i == B_PF || i == B_PF + 1;
    mbar_init(smem_u32(&sm->bar[i]), by_softmax ? (uint32_t)kWarps : k_empty || v_empty ? (k_empty ? 4u * KG : 0u) + (v_empty ? 4u : 0u) : by_four ? 4u : 1u);
    if (i == 0) sm->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Launched as a programmatic dependent: everything above touches no global memory; here the previous kernel's writes
  // become visible.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (not before: the kernels that this one waits for may still want tensor memory)
  if (warp == kWarpQK) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem)),
                 "n"(K::kTmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // units per CTA; extra >= 0: every segment has CTAs of its own, its draft tile counting 1 + extra units
  const int per = sm->per, extra = sm->extra;
  const int total = sm->cum[bd.batch];
  const int u_begin = min(total, (int)blockIdx.x * per), u_end = min(total, u_begin + per);
  if (blockIdx.x == 0) {   // for the merge
#pragma unroll 1
    for (int i = tid; i <= bd.batch; i += kAllThreads) p.cum[i] = sm->cum[i];
    if (tid == 0) { p.cum[kMaxBatch + 1] = per; p.cum[kMaxBatch + 2] = extra; }
  }
  // The piece that begins at unit u.
  auto piece_at = [&](int u) {
    Piece pc;
    int lo = 0;      // sequences that end at or before u
#pragma unroll 1
    for (int b = 0; b < bd.batch; b += 32) {
      const bool before = b + lane < bd.batch - 1 && sm->cum[b + lane + 1] <= u;
      const int n = __popc(__ballot_sync(0xffffffffu, before));
      lo += n;
      if (n < 32) break;
    }
    const int line = (sm->cum[lo + 1] - sm->cum[lo]) / parts;     // units of one of the sequence's segments
    const int rem = u - sm->cum[lo], s = rem / line, at = rem - s * line;
    pc.b = lo;
    pc.g = p.hparts == 1 ? s : s / p.hparts;
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
    // the same for every lane, and known to be (all nine of them shuffled: 64 sequences 388 us against 383)
    pc.first = __shfl_sync(0xffffffffu, pc.first, 0);
    pc.tiles = __shfl_sync(0xffffffffu, pc.tiles, 0);
    pc.span = __shfl_sync(0xffffffffu, pc.span, 0);
    return pc;
  };
  const uint32_t bars = smem_u32(&sm->bar[0]);
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto wait = [&](int i, int n) { return wait4(bar(i), (uint32_t)n & 1u, &sm->abort); };
  // The softmax warps do not leave early: after an expired wait no other one waits, and they run through, so that
  // their named barriers always find all of them.
  auto spin = [&](int i, int n) {
    wait(i, n);
    __syncwarp();
  };
  const uint32_t tmem = sm->tmem;

  // Positions in the rings, counted along: an index and the parity of its round.
  struct Ring {
    int at = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next(int n) {
      if (++at == n) { at = 0; round ^= 1u; }
    }
  };
  // A ring for each group of widening warps, `size` barriers apart.
  struct Rings {
    Ring of[WG];
    __device__ __forceinline__ Ring get(int g) const { return WG == 2 && g ? of[WG - 1] : of[0]; }
    __device__ __forceinline__ void next(int g, int n) {
      if (WG == 2 && g) of[WG - 1].next(n); else of[0].next(n);
    }
  };
  auto wait_full = [&](int first, const Ring& r) { return wait(first + r.at, (int)r.round); };
  auto wait_empty = [&](int first, const Ring& r) { return wait(first + r.at, (int)r.round ^ 1); };
  // A position that some query sees: from the root's oldest visible one on.
  auto first_seen = [&](int L) { return p.window > 0 ? L - p.window + 1 : 0; };

  if (warp >= kWarpK) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(K::kRegsRest));
    if (warp <= kWarpV) {
      // ---------------------------------------------------------- producers (where the ring is joint, the first alone)
      // Page ids come a group of four tiles at a time (lane l: page l % 8 of the group's l / 8), two groups ahead of
      // their use: under a full memory system a load takes as long as a tile or two.
      const bool is_k = warp == kWarpK;
      constexpr uint32_t kBytes = K::kPageStride;     // of a page
      const int n_ring = is_k ? KS : VS, b_full = is_k ? B_KF : B_VF, b_empty = is_k ? B_KE : B_VE;
      uint8_t* const buf = is_k ? sK : sV;
      const uint64_t policy = l2_evict_first();
      Rings rings;
      int turn = 0;      // whose tile it is
      bool ok = is_k || !K::kJoint;
#pragma unroll 1
      for (int u = u_begin; u < u_end && ok;) {
        const Piece pc = piece_at(u);
        u += pc.span;
        const int* row = p.page_table + (size_t)pc.b * p.max_pages;
        const int left = pc.tiles - (pc.first == 0 ? 1 : 0);      // the draft tile does not come from the cache
        if (pc.first == 0) turn = turn + 1 == WG ? 0 : turn + 1;
        const int t0 = pc.t0(max(pc.first, 1));
        const uint8_t* src = p.cache + (size_t)(2 * pc.g + (is_k ? 0 : 1)) * K::kRecord;
        const size_t page_bytes = (size_t)p.hkv * 2 * K::kRecord;
        auto ids_from = [&](int n) {     // of the piece's context tiles n .. n + 3
          const int t = t0 - (n + (lane >> 3)) * kTile + (lane & 7) * kPage;
          return n + (lane >> 3) < left && t < pc.L ? row[t / kPage] : -1;
        };
        int ids_next = ids_from(0), ids_after = ids_from(4), ids = -1;
        uint32_t good = 0;    // pages of the group that can be loaded
#pragma unroll 1
        for (int n = 0; n < left; ++n) {
          const int sub = (n & 3) * 8;
          if (sub == 0) {
            ids = ids_next;
            ids_next = ids_after;
            ids_after = ids_from(n + 8);
            const bool in_pool = (unsigned)ids < (unsigned)p.num_pool_pages;
            good = __ballot_sync(0xffffffffu, in_pool);
            if (is_k) {
              const int at = t0 - (n + (lane >> 3)) * kTile + (lane & 7) * kPage;
              if (n + (lane >> 3) < left && at < pc.L && at + kPage > first_seen(pc.L) && !in_pool)
                report(p.dev_status, SD_DEV_BAD_PAGE);
            }
          }
          const int valid = min(kTile, pc.L - (t0 - n * kTile));
          const uint32_t need = (1u << ((valid + kPage - 1) / kPage)) - 1u;
          const uint32_t have = (good >> sub) & need;
          const Ring ring = rings.get(turn);
          const int at = turn * n_ring + ring.at;
          ok = __all_sync(0xffffffffu, wait_empty(b_empty + turn * n_ring, ring));
          if (!ok) break;
          uint8_t* dst = buf + at * K::kSlotBytes;
          if (need != have) {   // ids out of range count as zeros: scales of 0
#pragma unroll 1
            for (int e = lane; e < 8 * (int)(kBytes / 16); e += 32)
              if (((need & ~have) >> (e / (kBytes / 16))) & 1u) reinterpret_cast<uint4*>(dst)[e] = make_uint4(0, 0, 0, 0);
            fence_async_smem();   // the slot's next contents come by another path
            __syncwarp();
          }
          int page[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) page[j] = __shfl_sync(0xffffffffu, ids, sub + j);
          if (elect_one()) {
            const uint32_t full = bar(b_full + at), to = smem_u32(dst);
            mbar_expect_tx(full, (uint32_t)__popc(have) * kBytes);
            if (have == 0xffu) {
#pragma unroll
              for (int j = 0; j < 8; ++j) bulk_record(to + j * kBytes, src + (size_t)page[j] * page_bytes, kBytes, full, policy);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if ((have >> j) & 1u) bulk_record(to + j * kBytes, src + (size_t)page[j] * page_bytes, kBytes, full, policy);
            }
          }
          __syncwarp();
          rings.next(turn, n_ring);
          turn = turn + 1 == WG ? 0 : turn + 1;
        }
      }
      // After an abort no copy may still be landing when the CTA ends: wait, bounded, for both rounds of every slot.
      if (lane == 0 && *(volatile int*)&sm->abort) {
#pragma unroll 1
        for (int s = 0; s < 2 * n_ring * WG; ++s) {
          const long long begin = clock64();
          while (!mbar_test(bar(b_full + (s >> 1)), (uint32_t)s & 1u) && clock64() - begin < kWaitCycles / 64) {
          }
        }
      }
    } else if (warp == kWarpQK) {
      // ---------------------------------------------------------- QK issuer
      Ring s_ring;
      int np = 0, it = 0, turn = 0;
      uint32_t phase = 0;            // of a group's slots: a bit each
      bool ok = true;
      const uint64_t q_desc = sw128_desc(smem_u32(sQ), 16, 1024);
#pragma unroll 1
      for (int u = u_begin; u < u_end && ok; ++np) {
        const Piece pc = piece_at(u);
        u += pc.span;
        const int n_nodes = bd.q_indptr[pc.b + 1] - bd.q_indptr[pc.b];
        const int nq = (min(p.hpc, p.group - pc.c * p.hpc) * n_nodes + 15) & ~15;
        const uint32_t idesc = f16_idesc(128, nq, 0, 0);
        ok = __all_sync(0xffffffffu, wait(B_Q, np));
        const int end = pc.first + pc.tiles;
#pragma unroll 1
        for (int i = pc.first, n; i < end && ok; i += n) {
          n = min(T, end - i);
          ok = __all_sync(0xffffffffu, wait_empty(B_SE, s_ring));
          uint32_t d = tmem + s_ring.at * T * NQ;
#pragma unroll 1
          for (int j = 0; j < n && ok; ++j, d += NQ) {
            const uint32_t a0 = tmem + K::kColA + turn * KA * K::kSlotCols;
            const uint32_t full = bar(B_AKF + turn * KA), empty = bar(B_AKE + turn * KA);
            const uint32_t odd = (phase >> turn) & 1u;
#pragma unroll 1
            for (int k = 0; k < K::KU; ++k) {
#pragma unroll
              for (int s = 0; s < KA; ++s) {
                wait4(full + 8 * s, K::KU % 2 == 0 ? k & 1 : odd ^ (k & 1), &sm->abort);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
                  // a 64-dim block of Q^T is NQ rows of 128 bytes
                  const int ks = k * KA + s;
                  const uint64_t b = q_desc + (SW >= 64 ? ks * (SW / 64) * (NQ * 128 >> 4) : (ks >> 1) * (NQ * 128 >> 4) + (ks & 1) * 4);
#pragma unroll
                  for (int kk = 0; kk < SW / 16; ++kk) {
                    if (s > 0 || kk > 0)
                      umma_ta<1>(d, a0 + s * K::kSlotCols + kk * 8, b + (kk >> 2) * (NQ * 128 >> 4) + (kk & 3) * 2, idesc);
                    else
                      umma_ta<2>(d, a0, b, idesc, k > 0 ? 1u : 0u);
                  }
                  umma_commit(empty + 8 * s);
                  if (s == KA - 1 && k == K::KU - 1 && j == n - 1) umma_commit(bar(B_SF + (NS == 2 ? s_ring.at : it & 1)));
                }
                __syncwarp();
              }
            }
            ok = *(volatile int*)&sm->abort == 0;
            phase ^= 1u << turn;
            turn = turn + 1 == WG ? 0 : turn + 1;
          }
          s_ring.next(NS);
          ++it;
        }
      }
    } else {
      // ---------------------------------------------------------- PV issuer
      int it = 0, turn = 0;
      uint32_t phase = 0;
      bool ok = true;
      // P: 8-column chunks of T x 128 token rows x 16 bytes; MN-major without a swizzle
      const uint64_t p_desc0 = noswz_desc(smem_u32(sP), 128, T * kTile * 16);
      const uint64_t p_desc1 = noswz_desc(smem_u32(sP + K::kPBytes), 128, T * kTile * 16);
#pragma unroll 1
      for (int u = u_begin; u < u_end && ok;) {
        const Piece pc = piece_at(u);
        u += pc.span;
        const int n_nodes = bd.q_indptr[pc.b + 1] - bd.q_indptr[pc.b];
        const int nq = (min(p.hpc, p.group - pc.c * p.hpc) * n_nodes + 15) & ~15;
        const uint32_t idesc = f16_idesc(128, nq, 0, 1);
        const int end = pc.first + pc.tiles;
#pragma unroll 1
        for (int i = pc.first, n; i < end && ok; i += n, ++it) {
          n = min(T, end - i);
          ok = __all_sync(0xffffffffu, wait(B_PF + (it & 1), it >> 1));
          // With one S buffer the next QK has waited for the same softmax, and the softmax waits for it: it goes first, and this
          // PV beside that softmax.  (Two barriers in turn, so that the one after the next cannot complete unseen: its
          // softmax needs this PV.)
          if (NS == 1 && i + n < end) ok = __all_sync(0xffffffffu, wait(B_SF + ((it + 1) & 1), (it + 1) >> 1)) && ok;
          uint64_t b = it & 1 ? p_desc1 : p_desc0;
#pragma unroll 1
          for (int j = 0; j < n && ok; ++j, b += kTile) {
            const int valid = i + j == 0 ? n_nodes : min(kTile, pc.L - pc.t0(i + j));
            const uint32_t fresh = i == pc.first && j == 0 ? 0u : 1u;       // the piece's first products overwrite O
            const uint32_t a0 = tmem + K::kColA + (KA * WG + turn * VA) * K::kSlotCols;
            const uint32_t full = bar(B_AVF + turn * VA), empty = bar(B_AVE + turn * VA);
            const uint32_t odd = (phase >> turn) & 1u;
#pragma unroll 1
            for (int k = 0; k < K::VU; ++k) {
#pragma unroll
              for (int s = 0; s < VA; ++s) {
                wait4(full + 8 * s, K::VU % 2 == 0 ? k & 1 : odd ^ (k & 1), &sm->abort);
                __syncwarp();
                tc_fence_after();
                // slot k VA + s: 128-dim block mb of SW tokens
                const int mb = (k * VA + s) % MH, ts = (k * VA + s) / MH;
                const uint32_t d = tmem + K::kColO + mb * NQ, a = a0 + s * K::kSlotCols;
                const int steps = (valid - ts * SW + 15) / 16;      // of 16 tokens that hold any
                if (elect_one()) {
                  const uint64_t bb = b + ts * SW;
                  if (steps >= SW / 16) {
                    umma_ta<2>(d, a, bb, idesc, ts > 0 ? 1u : fresh);
#pragma unroll
                    for (int kk = 1; kk < SW / 16; ++kk) umma_ta<1>(d, a + kk * 8, bb + kk * 16, idesc);
                  } else {
#pragma unroll 1
                    for (int kk = 0; kk < steps; ++kk) umma_ta<2>(d, a + kk * 8, bb + kk * 16, idesc, ts > 0 || kk > 0 ? 1u : fresh);
                  }
                  umma_commit(empty + 8 * s);
                }
                __syncwarp();
              }
            }
            ok = *(volatile int*)&sm->abort == 0;
            phase ^= 1u << turn;
            turn = turn + 1 == WG ? 0 : turn + 1;
          }
          if (ok && elect_one()) umma_commit(bar(B_OD + (it & 1)));
          __syncwarp();
        }
      }
    }
  } else if (warp >= kWarpWideK) {
    // ------------------------------------------------------------ the widening warps
    // After an expired wait no other one waits, and they run through.
    if (K::kRegsWide < K::kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(K::kRegsWide));
    const bool is_k = warp < kWarpWideV;
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const int of_four = (warp - (is_k ? kWarpWideK : kWarpWideV)) >> 2;
    const int group = is_k ? of_four / KG : of_four, part = is_k ? of_four % KG : 0;     // whose tiles, and which slot of K's
    const uint32_t a_base = tmem + ((uint32_t)(quarter * 32) << 16) + K::kColA + (is_k ? group * KA : KA * WG + group * VA) * K::kSlotCols;
    const uint32_t a_full = bar(is_k ? B_AKF + group * KA : B_AVF + group * VA), a_empty = bar(is_k ? B_AKE + group * KA : B_AVE + group * VA);
    const int n_ring = is_k ? KS : VS, b_full = (is_k ? B_KF : B_VF) + group * n_ring, b_empty = (is_k ? B_KE : B_VE) + group * n_ring;
    const uint8_t* const buf = (is_k ? sK : sV) + group * n_ring * K::kSlotBytes;
    Ring ring;
    uint32_t odd = 0;             // parity of the group's tiles
    auto slot_free = [&](int s, uint32_t parity) {
      wait4(a_empty + 8 * s, parity ^ 1u, &sm->abort);
      __syncwarp();
      tc_fence_after();
    };
    // A slot's lanes are stored: to the issuer.
    auto slot_done = [&](int s) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full + 8 * s);
    };
    int turn = 0;      // whose turn the tile is
#pragma unroll 1
    for (int u = u_begin; u < u_end;) {
      const Piece pc = piece_at(u);
      u += pc.span;
      const int q0 = bd.q_indptr[pc.b], n_nodes = bd.q_indptr[pc.b + 1] - q0;
      const int seen = first_seen(pc.L);
#pragma unroll 1
      for (int i = pc.first; i < pc.first + pc.tiles; ++i) {
        const bool draft = i == 0, mine = turn == group;
        turn = turn + 1 == WG ? 0 : turn + 1;
        if (!mine) continue;
        if (draft) {
          // the draft block, bf16 as it is (what is no number there goes through the scores: zeros here, see `wild`)
#pragma unroll 1
          for (int n = 0; n < (is_k ? K::KU * KA : K::VU * VA); ++n) {
            const int s = n % (is_k ? KA : VA), k = n / (is_k ? KA : VA);
            if (KG == 2 && is_k && s != part) continue;
            slot_free(s, (is_k ? K::KU : K::VU) % 2 == 0 ? k & 1 : odd ^ (k & 1));
            if (is_k) {
              const uint4* src = reinterpret_cast<const uint4*>(p.k_new + (long long)(q0 + min(row, n_nodes - 1)) * p.k_stride + pc.g * D);
#pragma unroll 1
              for (int h = 0; h < SW / 32; ++h) {
                uint32_t x[16];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint4 v = make_uint4(0, 0, 0, 0);
                  if (row < n_nodes) v = __ldg(src + (n * SW + h * 32) / 8 + e);
                  x[4 * e] = v.x; x[4 * e + 1] = v.y; x[4 * e + 2] = v.z; x[4 * e + 3] = v.w;
                }
                tmem_st16u(a_base + s * K::kSlotCols + h * 16, x);
              }
            } else {
              const int ts = n / MH, mb = n % MH;
              const uint16_t* src = reinterpret_cast<const uint16_t*>(p.v_new) + (long long)q0 * p.v_stride + pc.g * D + mb * 128 + row;
#pragma unroll 1
              for (int h = 0; h < SW / 32 && ts * SW + h * 32 < n_nodes; ++h) {
                uint32_t x[16];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const int r = ts * SW + h * 32 + e;
                  uint32_t v = 0;
                  if (r < n_nodes) v = __ldg(src + (long long)r * p.v_stride);
                  if ((v & 0x7f80u) == 0x7f80u) v = 0;
                  x[e >> 1] = e & 1 ? x[e >> 1] | v << 16 : v;
                }
                tmem_st16u(a_base + s * K::kSlotCols + h * 16, x);
              }
            }
            slot_done(s);
          }
          odd ^= 1u;
          continue;
        }
        const int t0 = pc.t0(i);
        wait_full(b_full, ring);
        __syncwarp();
        if (is_k) {
          // this thread's token, block after block of 32 dims (rolled: the roles' loops share an instruction cache)
          const uint8_t* rec = buf + ring.at * K::kSlotBytes + (row >> 4) * K::kPageStride;
          const uint8_t* words = rec + (row & 15) * 16;
          uint16_t* sc = reinterpret_cast<uint16_t*>(const_cast<uint8_t*>(rec) + kv4_codes(D) + (row & 15) * (D / 16));
          // of this group's blocks: with bits that do not count, or beyond the largest
          static_assert(KG == 1 || SW == 32, "every second block");
          auto mine_of = [&](int e) {      // blocks 2 e and 2 e + 1
            return KG == 1 ? ~0u : 0xffffu << (16 * part);
          };
          bool odd_scale = false;
#pragma unroll
          for (int e = 0; e < D / 64; ++e) {
            const uint32_t two = reinterpret_cast<const uint32_t*>(sc)[e] & mine_of(e), most = kKv4BadScale - 1u | (kKv4BadScale - 1u) << 16;
            odd_scale |= (two & 0x00070007u) != 0u || __vmaxu2(two & 0x7fff7fffu, most) != most;
          }
          if (odd_scale) {             // rare: put right in place (nobody else reads these)
            bool bad = false;
#pragma unroll 1
            for (int e = 0; e < D / 32; ++e) {
              if ((mine_of(e >> 1) >> (16 * (e & 1)) & 1u) == 0u) continue;
              sc[e] = (uint16_t)kv4_sane(sc[e], bad);
            }
            fence_async_smem();
            if (bad && t0 + row < pc.L && t0 + row >= seen) report(p.dev_status, SD_DEV_BAD_SCALE);
          }
          if (KG == 2) {
            words += part * (SW / 32) * (kPage * 16);
            sc += part * (SW / 32);
          }
#pragma unroll 1
          for (int n = KG == 2 ? part : 0; n < K::KU * KA; n += KG) {
            const int s = n % KA, k = n / KA;
            const uint32_t to = a_base + s * K::kSlotCols;
            if (!K::kEarly) slot_free(s, K::KU % 2 == 0 ? k & 1 : odd ^ (k & 1));
#pragma unroll 1
            for (int h = 0; h < SW / 32; ++h) {
              const uint4 w = *reinterpret_cast<const uint4*>(words);
              const __nv_bfloat162 sv = kv4_scale2(__byte_perm(*sc, 0, 0x1010)), less = kv4_less(sv);
              words += kPage * 16;
              ++sc;
              const uint32_t* ww = reinterpret_cast<const uint32_t*>(&w);
              uint32_t x[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = kv4_pair(ww[e >> 2], e & 3, sv, less);
              if (K::kEarly && h == 0) slot_free(s, K::KU % 2 == 0 ? k & 1 : odd ^ (k & 1));
              tmem_st16u(to + h * 16, x);
            }
            if (KG == 2) {
              words += (KG - 1) * (SW / 32) * (kPage * 16);
              sc += (KG - 1) * (SW / 32);
            }
            slot_done(s);
          }
        } else {
          // this thread's dim (of each 128): the scales of its block of 32, token pair by token pair, are the warp's
          const uint8_t* pages = buf + ring.at * K::kSlotBytes;
          const bool plain = t0 >= seen && t0 + kTile <= pc.L;
          uint2* const vs = sm->vs[group * 4 + quarter][0];
#pragma unroll
          for (int r = 0; r < 2 * MH; ++r) {
            const int mb = r >> 1, pair = (r & 1) * 32 + lane;
            uint32_t s2 = *reinterpret_cast<const uint32_t*>(pages + (pair >> 3) * K::kPageStride + kv4_codes(D) +
                                                             (mb * 4 + quarter) * 32 + (pair & 7) * 4);
            s2 &= kKv4ScaleBits | kKv4ScaleBits << 16;
            if (!plain) {
              // tokens that nobody sees count 0 (their records may hold anything)
              const int t = t0 + 2 * pair;
              if (t >= pc.L || t < seen) s2 &= 0xffff0000u;
              if (t + 1 >= pc.L || t + 1 < seen) s2 &= 0x0000ffffu;
            }
            const uint32_t most = kKv4BadScale - 1u | (kKv4BadScale - 1u) << 16;
            if (__vmaxu2(s2 & 0x7fff7fffu, most) != most) {
              bool bad = false;
              s2 = kv4_sane(s2, bad);
              report(p.dev_status, SD_DEV_BAD_SCALE);
            }
            const __nv_bfloat162 less = kv4_less(kv4_scale2(s2));
            vs[mb * 64 + pair] = make_uint2(s2, *reinterpret_cast<const uint32_t*>(&less));
          }
          __syncwarp();
#pragma unroll 1
          for (int n = 0; n < K::VU * VA; ++n) {
            const int s = n % VA, k = n / VA, mb = n % MH, ts = n / MH;      // 128-dim block mb of SW tokens
            if (!K::kEarly) slot_free(s, K::VU % 2 == 0 ? k & 1 : odd ^ (k & 1));
            const uint8_t* words = pages + ts * (SW / 16) * K::kPageStride + (mb * 128 + row) * 8;
            const uint4* sl_at = reinterpret_cast<const uint4*>(vs + mb * 64 + ts * (SW / 2));
            const uint32_t to = a_base + s * K::kSlotCols;
#pragma unroll 1
            for (int h = 0; h < SW / 32; ++h, words += 2 * K::kPageStride, sl_at += 8) {
              const uint2 w0 = *reinterpret_cast<const uint2*>(words), w1 = *reinterpret_cast<const uint2*>(words + K::kPageStride);
              uint32_t x[16];
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const uint4 sl = sl_at[e >> 1];
                const uint32_t word = e & 8 ? (e & 4 ? w1.y : w1.x) : (e & 4 ? w0.y : w0.x);
                x[e] = kv4_pair(word, e & 3, kv4_scale2(sl.x), kv4_scale2(sl.y));
                x[e + 1] = kv4_pair(word, (e & 3) + 1, kv4_scale2(sl.z), kv4_scale2(sl.w));
              }
              if (K::kEarly && h == 0) slot_free(s, K::VU % 2 == 0 ? k & 1 : odd ^ (k & 1));
              tmem_st16u(to + h * 16, x);
            }
            slot_done(s);
          }
        }
        odd ^= 1u;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b_empty + ring.at));
        ring.next(n_ring);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warps
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(K::kRegsSoft));
    const int group = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;                       // token row of S; dim (mod 128) of O^T
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    auto sync_all = [] { asm volatile("bar.sync 7, %0;" ::"n"(kWarps * 32) : "memory"); };        // the softmax warps
    auto sync_group = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); };     // the group's four
    Ring s_ring;
    int it = 0;
#pragma unroll 1
    for (int u = u_begin; u < u_end;) {
      const Piece pc = piece_at(u);
      u += pc.span;
      const int q0 = bd.q_indptr[pc.b], n_nodes = bd.q_indptr[pc.b + 1] - q0;
      const int hpc = min(p.hpc, p.group - pc.c * p.hpc);
      const int head0 = pc.g * p.group + pc.c * p.hpc;
      const int rows = hpc * n_nodes, nc = (rows + 15) / 16;
      const int mine = min(CC, max(0, nc - group * CC)), c_first = group * CC;   // chunks of this group in use
      const int col0 = c_first * 16;
      const bool has_draft = pc.first == 0;
      // ---------------------------------------------------------- staging: Q and the tree
      // (the previous piece's products have all finished: its last scores and its last O were waited for)
      // the tree, where something goes by it: the draft block, a window's depths, a bias
      const bool needs_tree = has_draft || MOD || p.window > 0;
      if (needs_tree && tid < n_nodes) {
        const int up = p.parents[q0 + tid];
        sm->par[tid] = (int8_t)(up < -1 || up >= kMaxNodes ? -2 : up);
        sm->wild[tid] = 0;
      }
      {
        constexpr int LPR = D / 8, RPW = 32 / LPR;                     // lanes per row, rows per warp and load
        constexpr int U = (NQ + kWarps * RPW - 1) / (kWarps * RPW);    // a warp's query rows, RPW at a time
        constexpr int UB = U < 12 ? U : 12;                            // of them in flight
        const int sub = lane / LPR, ch = lane % LPR;                   // 8-value chunk of the row
        const int n_q = nc * 16;
        const float inv_hpc = 1.0f / (float)hpc;
#pragma unroll 1
        for (int i0 = 0; i0 < U; i0 += UB) {
          if ((i0 * kWarps + warp) * RPW >= n_q) break;
          uint4 x[UB];
#pragma unroll
          for (int i = 0; i < UB; ++i) {
            const int r = ((i0 + i) * kWarps + warp) * RPW + sub;
            const int node = __float2int_rz(((float)r + 0.5f) * inv_hpc);   // r / hpc, exact for r < 2^20
            x[i] = make_uint4(0, 0, 0, 0);
            if (r < rows)
              x[i] = __ldg(reinterpret_cast<const uint4*>(p.q + (long long)(q0 + node) * p.q_stride +
                                                          (head0 + r - node * hpc) * D) + ch);
          }
#pragma unroll
          for (int i = 0; i < UB; ++i) {
            const int r = ((i0 + i) * kWarps + warp) * RPW + sub;
            // a row with a NaN or an infinity: all NaN, and so its scores
            const uint32_t bad = __ballot_sync(0xffffffffu, wild8(x[i]));
            if (RPW == 1 ? bad != 0u : (bad >> (sub * LPR) & ((1ull << LPR) - 1ull)) != 0u)
              x[i] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            if (r < n_q)
              *reinterpret_cast<uint4*>(sQ + (ch >> 3) * NQ * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = x[i];
          }
        }
        sync_all();
        if (has_draft) {
#pragma unroll 1
          for (int r = warp * RPW + sub; r < 2 * n_nodes; r += kWarps * RPW) {
            const int n = r >> 1;
            const uint4 y = __ldg(reinterpret_cast<const uint4*>(
                (r & 1 ? p.v_new + (long long)(q0 + n) * p.v_stride : p.k_new + (long long)(q0 + n) * p.k_stride) + pc.g * D) + ch);
            if (wild8(y)) sm->wild[n] = 1;
          }
        }
      }
      fence_async_smem();
#pragma unroll 1
      for (int q = tid; q < NQ; q += kWarps * 32) {
        sm->m[q] = q < nc * 16 ? 0.f : -1e30f;     // no reference yet; columns past those in use: below everything
        if (MOD) sm->slope[q] = p.slopes != nullptr && q < rows ? p.slopes[head0 + q % hpc] * kLog2e : 0.f;
      }
      if (tid < 3) sm->large[tid] = 0;
      // the tree: root paths and depths
      if (needs_tree && tid < n_nodes) {
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
      }
      sync_all();
      if (tid == 0) mbar_arrive(bar(B_Q));
      if (has_draft && n_nodes > 1) {
        // While the first product runs: the root paths turned round by ballots, a row of the tile a turn.
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
      const int lo_root = first_seen(pc.L);
      const float fac = p.scale * kLog2e;
      // Until a tile that every column sees something of has passed, columns may have no reference.
      bool settled = false;
      // score times factor less reference is one fma, exact but for its one rounding; so what the maximum itself comes to is
      // what its product lost when it became the reference: up to 2^4 at references of 2^28, and beyond every exponent where
      // cache or queries are huge.  From kLarge on the product is rounded first, tile by tile: the maximum is 0 again.
      bool large = false;
      const int end = pc.first + pc.tiles;
#pragma unroll 1
      for (int i = pc.first, subs; i < end; i += subs, ++it) {
        const bool fresh = i == pc.first;
        subs = min(T, end - i);
        const bool band = p.window > 0 && pc.t0(i + subs - 1) < lo_root + kMaxNodes;
        const bool masked = i <= 1 && (i == 0 || pc.L - pc.t0(1) < kTile) || band;
        // Scores that are more than a multiple of the product are formed first and put back in its place.
        const bool formed = MOD || masked;
        const float mul = formed ? 1.f : fac;
        if (NS == 2) wait_full(B_SF, s_ring); else wait(B_SF + (it & 1), it >> 1);
        __syncwarp();
        tc_fence_after();
        const uint32_t s_addr = tmem + lane_addr + s_ring.at * T * NQ + col0;
        if (formed) {
#pragma unroll 1
          for (int j = 0; j < subs; ++j) {
            const bool draft = i + j == 0;
            const int t0 = pc.t0(i + j), valid = draft ? n_nodes : min(kTile, pc.L - t0);
            // Which columns see this row, one bit each.
            using Bits = typename BitsOf<CC>::type;
            Bits vis = row < valid && !draft && !band ? ~(Bits)0 : 0;
            if (row < valid && (draft || band)) {
              // node by node, from the one of the group's first column: its columns see this row, or none of them does
              int n = col0 / hpc, at = n * hpc - col0;       // the node's first column, less the group's
              const Bits full = ((Bits)1 << hpc) - 1;
              Bits bits = full >> -at;
              unsigned long long sees = draft && n < n_nodes ? sm->anc[row] >> n : 0ull;
#pragma unroll 1
              for (; at < CC * 16 && n < n_nodes; ++n, sees >>= 1) {
                vis |= (draft ? (sees & 1ull) != 0ull : t0 + row >= lo_root + sm->depth[n]) ? bits : (Bits)0;
                at += hpc;
                bits = full << (at & (8 * (int)sizeof(Bits) - 1));
              }
            }
            // the bias' distance is counted from the root: a node's depth shifts all its scores alike (see the log-sum-exp)
            const float rel = draft ? (row < n_nodes ? (float)sm->depth[row] : 0.f) : (float)(t0 + row - pc.L);
            const bool nan_row = draft && row < n_nodes && sm->wild[row] != 0;
#pragma unroll 1
            for (int c = 0; c < mine; ++c) {
              float a[16];
              tmem_ld16(s_addr + j * NQ + c * 16, a);
              tmem_wait_ld();
              if (MOD && p.softcap > 0.f) {
                // c tanh(x / c) = c - 2 c / (1 + 2^(2 log2e x / c))
                const float cl = p.softcap * kLog2e, ky = fac * p.cap_exp;
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const float2 y = mul2(make_float2(a[e], a[e + 1]), make_float2(ky, ky));
                  const float2 d = add2(make_float2(fast_exp2(y.x), fast_exp2(y.y)), make_float2(1.f, 1.f));
                  const float2 s = fma2(make_float2(fast_rcp(d.x), fast_rcp(d.y)), make_float2(-2.f * cl, -2.f * cl), make_float2(cl, cl));
                  a[e] = s.x;
                  a[e + 1] = s.y;
                }
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) a[e] *= fac;
              }
              if (MOD) {
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const float2 sl = *reinterpret_cast<const float2*>(&sm->slope[col0 + c * 16 + e]);
                  const float2 s = fma2(sl, make_float2(rel, rel), make_float2(a[e], a[e + 1]));
                  a[e] = s.x;
                  a[e + 1] = s.y;
                }
              }
              if (masked) {
                const uint32_t bits = (uint32_t)(vis >> (c * 16));
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float s = nan_row ? __int_as_float(0x7fc00000) : a[e];
                  a[e] = (bits >> e) & 1u ? s : -INFINITY;
                }
              }
              tmem_st16(s_addr + j * NQ + c * 16, a);
            }
          }
          tmem_wait_st();
        }
        // ---- the weights, on the assumption that no warp of the group has to move a reference; a chunk where one of this
        // warp's would pass 2^kRise waits for that
        uint32_t missed = 0;
        uint8_t* const p_row = sP + (it & 1) * K::kPBytes + c_first * 2 * T * kTile * 16 + row * 16;
        auto scored = [&](int c, float (&a)[16], float by) {     // exponents in place of the scores; their maximum
          float most = -INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 m = *reinterpret_cast<const float4*>(&sm->m[col0 + c * 16 + 4 * k]);
            const float2 d0 = fma2(make_float2(a[4 * k], a[4 * k + 1]), make_float2(by, by), make_float2(m.x, m.y));
            const float2 d1 = fma2(make_float2(a[4 * k + 2], a[4 * k + 3]), make_float2(by, by), make_float2(m.z, m.w));
            a[4 * k] = d0.x; a[4 * k + 1] = d0.y; a[4 * k + 2] = d1.x; a[4 * k + 3] = d1.y;
            most = fmaxf(fmaxf(most, fmaxf(d0.x, d0.y)), fmaxf(d1.x, d1.y));
          }
          return most;
        };
        auto weigh = [&](int j, int c, float (&d)[16]) {     // weights in place of the exponents, and into P
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            d[2 * k] = fast_exp2(d[2 * k]);
            d[2 * k + 1] = fast_exp2(d[2 * k + 1]);
            const __nv_bfloat162 h = __floats2bfloat162_rn(d[2 * k], d[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
          }
          uint8_t* at = p_row + j * kTile * 16 + c * 2 * T * kTile * 16;
          *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(at + T * kTile * 16) = make_uint4(w[4], w[5], w[6], w[7]);
        };
        auto add_up = [&](float2 (&total)[8], const float (&e)[16]) {
#pragma unroll
          for (int k = 0; k < 8; ++k) total[k] = add2(make_float2(e[2 * k], e[2 * k + 1]), total[k]);
        };
        const uint32_t all = (1u << mine) - 1u;
        // (into the buffer that the PV before the last has left)
        if (it >= 2) spin(B_OD + (it & 1), (it >> 1) - 1);
        if (settled && !large) {
          // (whether a chunk's weights count is asked when they are there)
#pragma unroll 1
          for (int j = 0; j < subs; ++j) {
#pragma unroll
            for (int c = 0; c < CC; ++c) {
              if (c >= mine) break;
              float x[16];
              tmem_ld16(s_addr + j * NQ + c * 16, x);
              wait_scores(x);
              const bool over = __any_sync(0xffffffffu, scored(c, x, mul) > kRise);
              weigh(j, c, x);
              if (over) missed |= 1u << (j * CC + c);
              else add_up(sum[c], x);
            }
          }
        } else {
          missed = 0xffffffffu;
        }
        // chunks of any tile
        uint32_t chunks = missed;
#pragma unroll
        for (int j = 1; j < T; ++j) chunks |= missed >> (j * CC);
        if (lane == 0) {
          sm->flag[group][it & 1][quarter] = (int)(chunks & all);
          mbar_arrive(bar(B_G + group));
        }
        settled = settled || i == 0 || !band;
        spin(B_G + group, it);
        const int4 fl = *reinterpret_cast<const int4*>(sm->flag[group][it & 1]);
        const uint32_t todo = (uint32_t)(fl.x | fl.y | fl.z | fl.w);     // chunks whose references move
        if (todo != 0u) {
          // The exact maxima of these chunks' columns and new references (unset ones are 0, set ones never are).
#pragma unroll
          for (int c = 0; c < CC; ++c) {
            if ((todo >> c) & 1u) {
              float mx = -INFINITY;
#pragma unroll 1
              for (int j = 0; j < subs; ++j) {
                float a[16];
                tmem_ld16(s_addr + j * NQ + c * 16, a);
                tmem_wait_ld();
                const float x = warp_max16(a, lane);
                mx = x != x ? x : fmaxf(mx, x);      // a column of NaN stays one
              }
              if (lane < 16) sm->red[quarter][col0 + c * 16 + lane] = mx * mul;
            }
          }
          sync_group();
          const int mine_col = quarter * 32 + lane, q = col0 + mine_col;
          if (mine_col < mine * 16 && ((todo >> (mine_col >> 4)) & 1u)) {
            const float old = -sm->m[q];
            const float mt = fmaxf(fmaxf(sm->red[0][q], sm->red[1][q]), fmaxf(sm->red[2][q], sm->red[3][q]));
            float now = mt == -INFINITY ? old : old == 0.f ? mt : fmaxf(old, mt);
            if (now == 0.f && mt != -INFINITY) now = 1e-30f;
            sm->alpha[q] = old == 0.f ? 1.f : fast_exp2(old - now);
            sm->m[q] = -now;
            if (fabsf(now) > kLarge) sm->large[group] = 1;
          }
          sync_group();
          large = sm->large[group] != 0;
          // O belongs to the previous tile's PV until it has finished
          if (!fresh) spin(B_OD + ((it - 1) & 1), (it - 1) >> 1);
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < CC; ++c) {
            if (!((todo >> c) & 1u)) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              sum[c][e] = mul2(sum[c][e], *reinterpret_cast<const float2*>(&sm->alpha[col0 + c * 16 + 2 * e]));
#pragma unroll 1
            for (int mb = 0; mb < (fresh ? 0 : MH); ++mb) {
              float v[16];
              const uint32_t ad = tmem + lane_addr + K::kColO + mb * NQ + col0 + c * 16;
              tmem_ld16(ad, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] *= sm->alpha[col0 + c * 16 + e];
              tmem_st16(ad, v);
            }
          }
          tmem_wait_st();
          // the weights of these chunks; sums have them already where this warp did not wait
#pragma unroll 1
          for (int j = 0; j < subs; ++j) {
#pragma unroll
            for (int c = 0; c < CC; ++c) {
              if (!((todo >> c) & 1u)) continue;
              float x[16];
              tmem_ld16(s_addr + j * NQ + c * 16, x);
              wait_scores(x);
              if (large) {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = __fmul_rn(x[e], mul);
              }
              scored(c, x, large ? 1.f : mul);
              weigh(j, c, x);
              if ((missed >> (j * CC + c)) & 1u) add_up(sum[c], x);
            }
          }
        }
        tc_fence_before();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_SE + s_ring.at));
          mbar_arrive(bar(B_PF + (it & 1)));
        }
        s_ring.next(NS);
      }

      // ---------------------------------------------------------- results
      // Column sums over the tile's 128 token rows: the lanes, then the quarters.
      sync_group();      // the last tile's readers of red[] are done
#pragma unroll
      for (int c = 0; c < CC; ++c) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) { v[2 * e] = sum[c][e].x; v[2 * e + 1] = sum[c][e].y; }
        const float s = warp_sum16(v, lane);
        if (lane < 16) sm->red[quarter][col0 + c * 16 + lane] = s;
      }
      sync_group();
      spin(B_OD + ((it - 1) & 1), (it - 1) >> 1);
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
        for (int mb = 0; mb < MH; ++mb) tmem_ld16(tmem + lane_addr + K::kColO + mb * NQ + col0 + c * 16, v[mb]);
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
