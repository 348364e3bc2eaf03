// Log probabilities of given tokens, entropy and top alternatives of logits
// rows (include/sd_logprobs.h: sd_logprobs).
//
// One pass over the logits.  A warp keeps the largest logit m that it has met, and each thread c, the number of its
// logits equal to m, s = sum e^d and w = sum e^d d over its other ones, d = (x - m) / T.  A larger m' turns s into
// a (s + c) and w into a (w + (m - m') / T (s + c)) with a = e^((m - m') / T), and c into 0.  Then
//   log S = log c + log1p(s / c),  lse = m / T + log S,  logprob = (x_t - m) / T - log S,  entropy = log S - w / (c + s):
// the terms at the maximum stand apart, so what the others add is kept to its own 24 bits, however small it
// is beside 1 (the log-probability of a near-certain token, and the entropy then, are nothing else).
// m rises in few tiles: the others pay one warp maximum for it.  Base 2 inside: d carries log2 e.
//
// Exponents are formed as x f - M, f = log2 e / T, M = m f rounded: one packed fma for two logits (with the difference first,
// and the type's own maxima, 12 instructions a logit became 8).  They are all off by r = m f - M, the exact
// remainder of an fma, which is put right in the sums: s by 2^-r, w by 2^-r (w - r s).
//
// Top.  A logit and its index make one 64-bit key that orders as they do (value, then
// the smaller index), so ties need no care and the `top` largest keys are one set.  A
// warp's 512 neighbouring logits are a segment, of which the stream keeps the maximum alone.  The `top` best segments by
// (maximum, then the smaller index) hold all of the set: what lies in another one has `top` maxima before it.
// They are looked through again (most of it comes from L2), for logits that reach a bar that `top` keys reach for certain:
// the last of those maxima, or the smallest over the warps of the ceil(top / warps)-th largest of the threads' maxima,
// whichever is more; of a segment `top` at most go on where more than 64 reach it.  (With a list and a bar that followed the stream, and a barrier for each 4096 logits, 2047 rows of
// 151936 with 20 alternatives took 217 us, now 132.)
//
// Bound by HBM for many rows without alternatives (1824 rows of 151936 bf16 logits 88 us, 0.93 of the copy rate); with 20 of
// them by what follows a row's stream, which the other three rows of an SM hide in part (115 us).  A fifth row
// would spill registers (92 -> 153 us).  Rows are cut into pieces over CTAs where there are few, and joined by a second
// launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace sdv {
namespace {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kPer = 16;                        // logits of a thread that are looked at together
constexpr int kGroup = kLpThreads * kPer;
constexpr int kSegment = 32 * kPer;             // logits that a warp looks at together
constexpr int kFew = 2 * kLpThreads;            // keys that are ranked one by one
constexpr int kListMax = 2048;
constexpr int kMaxGroups = kListMax / kLpWarps; // of a piece: a key for each segment fits the list
// 64 bytes of a thread are a tile, asked for while the tile before is looked at: 64 KB under way on an SM.
template <typename T>
constexpr int kLpTile = kLpThreads * 64 / (int)sizeof(T);
constexpr float kLog2eLp = 1.4426950408889634f;
using Key = unsigned long long;

__device__ __forceinline__ uint32_t order_of(float x) {   // larger floats, larger numbers; -0 as +0
  const uint32_t b = __float_as_uint(x + 0.f);
  return (int)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((int)o < 0 ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ Key key_of(float x, int v) { return (Key)order_of(x) << 32 | (uint32_t)~v; }

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN where either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {   // over the numbers
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// The terms against maximum m, which c of the logits have.
struct Stats {
  float m, c, s, w;
  __device__ __forceinline__ void rise(float to, float f) {      // f: log2(e) / T; to > m, m may be -inf (then all are 0)
    const float d = fmaxf((m - to) * f, -1e30f), a = fast_exp2(d), all = s + c;
    w = a * fmaf(d, all, w);
    s = a * all;
    c = 0.f;
    m = to;
  }
};

struct LpShared {
  Key list[kListMax];
  int n;             // keys in the list of segments, or of a join
  int found;         // keys of the segments' logits: a word of its own, as n is read where no barrier follows before this counts
  int segment[SD_LOGPROBS_MAX_TOP];
  int count;         // of a search
  uint32_t warp_bar[kLpWarps], thread_bar[kLpWarps];
  union {
    float top_of[kListMax];      // segments' maxima
    Key few[kFew];               // what a cut looks at
  };
  Key last[kLpWarps];
  float4 stats[kLpWarps];
};

// The j-th largest of o over the warp's lanes (0 where there are fewer).
__device__ __forceinline__ uint32_t warp_jth(uint32_t o, int j) {
  uint32_t best = 0u;
#pragma unroll 1
  for (int k = 0; k < j; ++k) {
    best = __reduce_max_sync(0xffffffffu, o);
    const uint32_t who = __ballot_sync(0xffffffffu, o == best);
    if ((int)(threadIdx.x & 31) == __ffs(who) - 1) o = 0u;
  }
  return best;
}

// The `top` largest of the list's n keys to its front, in descending order; all threads call it, n uniform.
// A key's place is the number of larger ones, so the keys are thinned out first: of the threads' largest keys (values
// alone), the j-th of each of W warps, j = ceil(top / W), and of these the smallest; `top` keys at least are no smaller.
// (Ranked as they were, the 380 that 38 pieces of a row leave took 8 us.)
__device__ __noinline__ void cut_list(LpShared& sh, int n, int top) {
  const int t = threadIdx.x;
  const Key* from_list = sh.list;
  if (n > 64) {
    Key most = 0;
#pragma unroll 1
    for (int i = t; i < n; i += kLpThreads) most = sh.list[i] > most ? sh.list[i] : most;
    const int full = min(kLpWarps, n >> 5), j = (top + full - 1) / full;     // warps whose threads all have a key
    const uint32_t jth = warp_jth((uint32_t)(most >> 32), j);
    if (t == 0) sh.count = 0;
    if ((t & 31) == 0) sh.warp_bar[t >> 5] = jth;
    __syncthreads();
    uint32_t value = sh.warp_bar[0];
#pragma unroll 1
    for (int w = 1; w < full; ++w) value = min(value, sh.warp_bar[w]);
    Key bar = (Key)value << 32;
    auto take = [&] {
#pragma unroll 1
      for (int i = t; i < n; i += kLpThreads) {
        const Key k = sh.list[i];
        if (k >= bar) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kFew) sh.few[at] = k;
        }
      }
      __syncthreads();
    };
    take();
    if (sh.count > kFew) {
      // many alike: the largest bar that leaves `top`, bit by bit (keys are distinct)
      bar = 0;
#pragma unroll 1
      for (int bit = 63; bit >= 0; --bit) {
        const Key with = bar | (Key)1 << bit;
        int mine = 0;
#pragma unroll 1
        for (int i = t; i < n; i += kLpThreads) mine += sh.list[i] >= with ? 1 : 0;
        __syncthreads();
        if (t == 0) sh.count = 0;
        __syncthreads();
        mine = __reduce_add_sync(0xffffffffu, mine);
        if ((t & 31) == 0 && mine != 0) atomicAdd(&sh.count, mine);
        __syncthreads();
        if (sh.count >= top) bar = with;
      }
      __syncthreads();
      if (t == 0) sh.count = 0;
      __syncthreads();
      take();
    }
    n = sh.count;
    from_list = sh.few;
  }
  // as many neighbouring threads a key as there are to spare
  int shift = 0;
  while (shift < 3 && n << (shift + 1) <= kLpThreads) ++shift;
  const int parts = 1 << shift, part = t & (parts - 1), step = (n + parts - 1) >> shift;
  const int begin = part * step, end = min(n, begin + step);
  Key mine[2];
  int larger[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = (t >> shift) + k * kLpThreads;
    mine[k] = i < n ? from_list[i] : 0;
    if (k > 0 && n <= kLpThreads) continue;
#pragma unroll 4
    for (int o = begin; o < end; ++o) larger[k] += from_list[o] > mine[k] ? 1 : 0;
    for (int d = 1; d < parts; d <<= 1) larger[k] += __shfl_xor_sync(0xffffffffu, larger[k], d);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (mine[k] != 0 && part == 0 && larger[k] < top) sh.list[larger[k]] = mine[k];
  __syncthreads();
}

// 16-byte pieces: as floats, their maximum (NaN where there is one), and no smaller than a bound (of the type, in each half
// of a word if it has two).
template <typename T>
struct Load;
template <>
struct Load<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ void put(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ float most_of(uint32_t a) { return __uint_as_float(a); }
  static __device__ __forceinline__ uint32_t bound(float lo) { return __float_as_uint(lo); }
  static __device__ __forceinline__ uint32_t above(uint32_t a, uint32_t lo) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(lo)));
  }
};
template <>
struct Load<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void put(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float most_of(uint32_t a) {
    return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t bound(float lo) {     // rounded down
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rd(lo)) * 0x10001u;
  }
  static __device__ __forceinline__ uint32_t above(uint32_t a, uint32_t lo) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(lo));
    return r;
  }
};
template <>
struct Load<__half> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float2 pair(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
  static __device__ __forceinline__ void put(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = pair(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float most_of(uint32_t a) { return max_nan(pair(a).x, pair(a).y); }
  static __device__ __forceinline__ uint32_t bound(float lo) { return (uint32_t)__half_as_ushort(__float2half_rd(lo)) * 0x10001u; }
  static __device__ __forceinline__ uint32_t above(uint32_t a, uint32_t lo) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(lo));
    return r;
  }
};
template <typename T>
__device__ __forceinline__ float value_of(T x) { return static_cast<float>(x); }

// A row's t-th given token (one a thread; -1: none), and its logit; -infinity where it is none.
static_assert(SD_LOGPROBS_MAX_GIVEN <= kLpThreads, "a thread for each given token");
__device__ __forceinline__ int given_token(const LogprobsParams& p, int row) {
  const int v = (int)threadIdx.x < p.given ? p.tokens[(size_t)row * p.given + threadIdx.x] : -1;
  return v < p.vocab ? v : -1;
}
template <typename T>
__device__ __forceinline__ T logit_of(const LogprobsParams& p, int row, int token) {
  return token >= 0 ? static_cast<const T*>(p.logits)[(long long)row * p.row_stride + token] : static_cast<T>(-INFINITY);
}

// A row's results from its statistics and (in sh.list, descending) its top keys.
template <typename T>
__device__ void finish_row(const LogprobsParams& p, const LpShared& sh, int row, Stats st, bool bad, float given) {
  const int t = threadIdx.x;
  const bool none = st.c == 0.f;      // nothing but -infinity
  const float log_s = bad ? NAN : none ? -INFINITY : logf(st.c) + log1pf(st.s / st.c);
  const float m = bad ? 0.f : st.m;
  auto logprob = [&](float x) { return bad ? NAN : x == -INFINITY ? -INFINITY : (x - m) * p.inv_t - log_s; };
  if (t == 0) {
    if (bad) report(p.dev_status, SD_DEV_NAN_LOGITS);
    if (p.lse != nullptr) p.lse[row] = bad ? NAN : none ? -INFINITY : m * p.inv_t + log_s;
    if (p.entropy != nullptr) p.entropy[row] = bad ? NAN : none ? 0.f : log_s - st.w / (st.c + st.s) * kLn2;
  }
  if (t < p.given) p.logprobs[(size_t)row * p.given + t] = logprob(given);
  for (int i = t; i < p.top; i += kLpThreads) {
    const size_t at = (size_t)row * p.top + i;
    const Key k = sh.list[i];
    p.top_ids[at] = bad ? -1 : (int)~(uint32_t)k;
    p.top_logprobs[at] = logprob(order_value((uint32_t)(k >> 32)));
  }
}

// Statistics over the warps, the same for every thread.
__device__ __forceinline__ Stats block_stats(LpShared& sh, Stats st, float f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float m = warp_max(st.m);
  if (st.m < m) st.rise(m, f);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    st.c += __shfl_xor_sync(0xffffffffu, st.c, d);
    st.s += __shfl_xor_sync(0xffffffffu, st.s, d);
    st.w += __shfl_xor_sync(0xffffffffu, st.w, d);
  }
  if (lane == 0) sh.stats[warp] = make_float4(m, st.c, st.s, st.w);
  __syncthreads();
  Stats all;
  all.m = -INFINITY;
  all.c = all.s = all.w = 0.f;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) all.m = fmaxf(all.m, sh.stats[w].x);
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
    const float4 o = sh.stats[w];
    Stats x;
    x.m = o.x; x.c = o.y; x.s = o.z; x.w = o.w;
    if (x.m < all.m) x.rise(all.m, f);
    all.c += x.c;
    all.s += x.s;
    all.w += x.w;
  }
  return all;
}

__device__ __forceinline__ float2 lp_fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 lp_add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

// The sums of tiles below the maximum, with exponents y f - M (see above), and what goes with that maximum.
struct Quick {
  float2 s, w;
  float less, r;        // -M; m f - M
  uint32_t lo;          // what counts for nothing counts as this, so that no exponent is infinite
  float floor;          // the same as a float
  bool on;
  __device__ __forceinline__ void clear() { s = w = make_float2(0.f, 0.f); }
  __device__ __forceinline__ void into(Stats& st) {
    if (on) {
      const float all = s.x + s.y, a = fast_exp2(-r);
      st.s = fmaf(a, all, st.s);
      st.w = fmaf(a, fmaf(-r, all, w.x + w.y), st.w);
    }
    clear();
  }
  template <typename T>
  __device__ __forceinline__ void none() {
    on = false;
    lo = Load<T>::bound(-INFINITY);
    floor = -INFINITY;
  }
  // far: 512 / f.  Not for maxima whose product with f is large (r would be), nor where the type has no number far enough
  // below.
  template <typename T>
  __device__ __forceinline__ void follow(float m, float f, float far) {
    less = -(m * f);
    r = fmaf(m, f, less);
    lo = Load<T>::bound(m - far);
    float y[Load<T>::kVec];
    Load<T>::put(make_uint4(lo, lo, lo, lo), y);
    floor = y[0];
    on = fabsf(less) < 1048576.f && floor > -INFINITY && (m - floor) * f < 1e30f;
    if (!on) none<T>();
  }
};

// A warp's segment of which many logits are in question (sorted ones, or many alike): of those that `pass` marks (a bit each of a
// lane's, value j * kVec + k at v + j * 32 * kVec + k) the `top` largest, of equal ones the first.  The largest number that as
// many reach is found bit by bit.  (Not in line: it would cost the stream its registers.)
template <typename T>
__device__ __noinline__ uint32_t segment_top(const T* x, int v, uint32_t pass, int top) {
  constexpr int kVec = Load<T>::kVec;
  const int lane = threadIdx.x & 31;
  uint32_t o[kPer], least = 0u;
#pragma unroll
  for (int e = 0; e < kPer; ++e) o[e] = (pass >> e) & 1u ? order_of(value_of(x[v + e / kVec * (32 * kVec) + e % kVec])) : 0u;
#pragma unroll 1
  for (uint32_t bit = 0x80000000u; bit != 0u; bit >>= 1) {
    const uint32_t with = least | bit;
    int more = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) more += o[e] >= with ? 1 : 0;
    if (__reduce_add_sync(0xffffffffu, more) >= top) least = with;
  }
  uint32_t equal = 0u;
  pass = 0u;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    pass |= o[e] > least ? 1u << e : 0u;
    equal |= o[e] == least ? 1u << e : 0u;
  }
  int left = top - __reduce_add_sync(0xffffffffu, __popc(pass));
#pragma unroll 1
  for (int j = 0; j < kPer / kVec; ++j) {
    uint32_t here = equal >> (j * kVec) & ((1u << kVec) - 1u);
    const int n = __popc(here);
    int upto = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += up;
    }
    int mine = left - (upto - n);      // of the equal ones, for this lane and those behind it
    for (; here != 0u && mine > 0; here &= here - 1u, --mine) pass |= (here & (0u - here)) << (j * kVec);
    left -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return pass;
}

// VEC: the rows start on 16 bytes and so does every 16-byte piece of them.
template <typename T, bool TOP, bool VEC>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_piece_kernel(const LogprobsParams p) {
  __shared__ LpShared sh;
  constexpr int kVec = Load<T>::kVec, kTile = kLpTile<T>, kPieces = kPer / kVec, kGroups = kTile / kGroup;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int row = blockIdx.x / p.pieces, piece = blockIdx.x - row * p.pieces;
  const T* x = static_cast<const T*>(p.logits) + (long long)row * p.row_stride;
  const int begin = piece * p.piece, end = min(p.vocab, begin + p.piece);
  const float f = p.inv_t * kLog2eLp, far = 512.f / f;
  pdl_wait();
  Stats st;
  st.m = -INFINITY;
  st.c = st.s = st.w = 0.f;
  Quick quick;
  quick.clear();
  quick.none<T>();
  float most = -INFINITY;      // of this thread
  bool bad = false;
  // A 16-byte piece; what lies past the end counts as tokens that cannot come.
  auto piece_at = [&](int v) {
    if (VEC && v + kVec <= end) return __ldcs(reinterpret_cast<const uint4*>(x + v));
    alignas(16) T e[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) e[k] = v + k < end ? x[v + k] : static_cast<T>(-INFINITY);
    return *reinterpret_cast<const uint4*>(e);
  };
  // A thread's logits of a tile: of its warp's segment in each group, kPieces pieces; a group's are asked for when those of
  // the tile before it have become floats.
  uint4 raw[4];
  int from = begin + warp * kSegment + lane * kVec;      // of the pieces that are asked for next
  auto fetch = [&](int g) {
    if (VEC && from + (g * kGroup + (kPieces - 1) * 32 * kVec + kVec) <= end) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        raw[g * kPieces + j] = __ldcs(reinterpret_cast<const uint4*>(x + from) + (g * kGroup / kVec + j * 32));
    } else {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) raw[g * kPieces + j] = piece_at(from + g * kGroup + j * 32 * kVec);
    }
  };
  // Where a row is one long stream, the tile after the next is asked for into L2, as the registers hold one (2047 rows of
  // 151936 144 -> 131 us; four tiles on 132; rows in pieces gain nothing).
  auto ahead = [&](int at) {
    if (VEC && p.pieces == 1 && t == 0 && at < end) {
      const uint32_t bytes = (uint32_t)min(kTile, end - at) * (uint32_t)sizeof(T) & ~15u;
      if (bytes > 0u) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(x + at), "r"(bytes) : "memory");
    }
  };
#pragma unroll
  for (int g = 0; g < kGroups; ++g) fetch(g);
  ahead(begin + kTile);
  const int token = p.pieces == 1 ? given_token(p, row) : -1;      // (its logit: once the stream is over)
#pragma unroll 1
  for (int tile = begin; tile < end; tile += kTile) {
    from += kTile;
    ahead(tile + 2 * kTile);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int at = tile + g * kGroup + warp * kSegment;
      if (at >= end) break;
      uint32_t big = raw[g * kPieces].x;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const uint4 v = raw[g * kPieces + j];
        big = Load<T>::most(Load<T>::most(Load<T>::most(big, v.x), Load<T>::most(v.y, v.z)), v.w);
      }
      const float top = Load<T>::most_of(big);
      bad |= top != top;
      const float warp_top = warp_max(top);
      if (TOP) {
        most = fmaxf(most, top);
        if (lane == 0) sh.top_of[(at - begin) / kSegment] = warp_top;
      }
      if (warp_top > st.m) {
        quick.into(st);
        st.rise(warp_top, f);
        quick.follow<T>(warp_top, f, far);
        bad |= warp_top == INFINITY;
      }
      float y[kPer];
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const uint4 v = raw[g * kPieces + j];
        Load<T>::put(make_uint4(Load<T>::above(v.x, quick.lo), Load<T>::above(v.y, quick.lo), Load<T>::above(v.z, quick.lo),
                                Load<T>::above(v.w, quick.lo)), y + j * kVec);
      }
      if (tile + kTile < end) fetch(g);
      if (warp_top == st.m && warp_top > -INFINITY) {
        float c = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const bool at_top = y[e] == st.m;
          c += at_top ? 1.f : 0.f;
          y[e] = at_top ? quick.floor : y[e];
        }
        st.c += c;
      }
      if (quick.on) {
        float2 sum = make_float2(0.f, 0.f), w = sum;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
          const float2 d = lp_fma2(make_float2(y[e], y[e + 1]), make_float2(f, f), make_float2(quick.less, quick.less));
          const float2 a = make_float2(fast_exp2(d.x), fast_exp2(d.y));
          sum = lp_add2(sum, a);
          w = lp_fma2(a, d, w);
        }
        quick.s = lp_add2(quick.s, sum);
        quick.w = lp_add2(quick.w, w);
      } else if (st.m > -INFINITY) {
        // rare; d is kept finite, so that the product is 0 where e^d is
        float sum = 0.f, w = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const float d = fmaxf((y[e] - st.m) * f, -1e30f), a = fast_exp2(d);
          sum += a;
          w = fmaf(a, d, w);
        }
        st.s += sum;
        st.w += w;
      }
    }
  }
  const T given = logit_of<T>(p, row, token);
  quick.into(st);
  if (TOP) {
    const int segments = (end - begin + kSegment - 1) / kSegment;
    // a bar from the threads' maxima, of the warps whose threads all have logits (the first in any case): `top` of them at
    // least are no smaller, or it is -infinity
    const int full = max(1, min(kLpWarps, (end - begin) / kSegment));
    if (warp < full) {
      const uint32_t jth = warp_jth(most != most ? 0u : order_of(most), (p.top + full - 1) / full);
      if (lane == 0) sh.thread_bar[warp] = jth;
    }
    if (t == 0) sh.n = sh.found = 0;
    __syncthreads();
    uint32_t bar = sh.thread_bar[0];
#pragma unroll
    for (int w = 1; w < kLpWarps; ++w) bar = w < full ? min(bar, sh.thread_bar[w]) : bar;
    // the segments that reach it: about twice `top`, if not all the same
    for (int i = t; i < segments; i += kLpThreads) {
      const uint32_t o = order_of(sh.top_of[i]);
      if (o >= bar) sh.list[atomicAdd(&sh.n, 1)] = (Key)o << 32 | (uint32_t)~i;
    }
    __syncthreads();
    int taken = sh.n;
    if (taken > p.top) {
      cut_list(sh, taken, p.top);
      taken = p.top;
      bar = max(bar, (uint32_t)(sh.list[p.top - 1] >> 32));
    }
    if (t < taken) sh.segment[t] = (int)~(uint32_t)sh.list[t];
    __syncthreads();
    const float reach = order_value(bar);
#pragma unroll 1
    for (int i = warp; i < taken; i += kLpWarps) {
      const int at = begin + sh.segment[i] * kSegment + lane * kVec;
      uint32_t pass = 0;       // this lane's logits that reach the bar, a bit each
      float y[kPer];
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int v = at + j * 32 * kVec;
        Load<T>::put(piece_at(v), y + j * kVec);
#pragma unroll
        for (int k = 0; k < kVec; ++k) pass |= y[j * kVec + k] >= reach ? 1u << (j * kVec + k) : 0u;
        if (v + kVec > end) pass &= ~(((1u << kVec) - 1u) << j * kVec) | (((1u << max(end - v, 0)) - 1u) << j * kVec);
      }
      auto key = [&](int e) {
        const int v = at + e / kVec * (32 * kVec) + e % kVec;
        return key_of(value_of(x[v]), v);
      };
      if (__reduce_add_sync(0xffffffffu, __popc(pass)) > 64) pass = segment_top<T>(x, at, pass, p.top);
#pragma unroll 1
      for (; pass != 0; pass &= pass - 1u) {
        const Key k = key(__ffs(pass) - 1);
        sh.list[atomicAdd(&sh.found, 1)] = k;
      }
      __syncwarp();
    }
    __syncthreads();
    const int n = sh.found;
    cut_list(sh, n, p.top);
    // a piece with fewer than `top` keys (the last of a row, or one with NaN): the rest sort behind everything
    for (int i = min(n, p.top) + t; i < p.top; i += kLpThreads) sh.list[i] = 0;
  }
  const bool any_bad = __syncthreads_or(bad ? 1 : 0) != 0;
  st = block_stats(sh, st, f);
  if (p.pieces == 1) {
    finish_row<T>(p, sh, row, st, any_bad, value_of(given));
  } else {
    if (t == 0) p.stats[blockIdx.x] = make_float4(st.m, any_bad ? NAN : st.c, st.s, st.w);
    if (TOP)
      for (int i = t; i < p.top; i += kLpThreads) p.keys[(size_t)blockIdx.x * p.top + i] = sh.list[i];
  }
}

// The pieces of a row joined: at most kMaxPieces of them.
constexpr int kMaxPieces = 64;
static_assert(kMaxPieces * SD_LOGPROBS_MAX_TOP <= kListMax && kMaxPieces <= kLpThreads, "a row's keys fit the list");

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_join_kernel(const LogprobsParams p) {
  __shared__ LpShared sh;
  const int row = blockIdx.x, t = threadIdx.x;
  const float f = p.inv_t * kLog2eLp;
  pdl_wait();
  const float given = value_of(logit_of<T>(p, row, given_token(p, row)));
  Stats st;
  st.m = -INFINITY;
  st.c = st.s = st.w = 0.f;
  bool bad = false;
  if (t < p.pieces) {
    const float4 v = p.stats[(size_t)row * p.pieces + t];
    st.m = v.x;
    bad = v.y != v.y;
    st.c = bad ? 0.f : v.y;
    st.s = v.z;
    st.w = v.w;
  }
  if (t == 0) sh.n = 0;
  __syncthreads();
  if (p.top > 0) {
    // a piece's last key has `top` keys of its own piece no smaller: the largest of these is a bar
    const Key* keys = p.keys + (size_t)row * p.pieces * p.top;
    const Key last = t < p.pieces ? keys[(size_t)t * p.top + p.top - 1] : 0;
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(last >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(last >> 32) == hi ? (uint32_t)last : 0u);
    if ((t & 31) == 0) sh.last[t >> 5] = (Key)hi << 32 | lo;
    __syncthreads();
    Key bar = 0;
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) bar = sh.last[w] > bar ? sh.last[w] : bar;
    for (int i = t; i < p.pieces * p.top; i += kLpThreads) {
      const Key k = keys[i];
      if (k != 0 && k >= bar) sh.list[atomicAdd(&sh.n, 1)] = k;
    }
  }
  bad = __syncthreads_or(bad ? 1 : 0) != 0;
  st = block_stats(sh, st, f);
  if (p.top > 0) {
    const int n = sh.n;
    __syncthreads();
    cut_list(sh, n, p.top);
  }
  finish_row<T>(p, sh, row, st, bad, given);
}

// Pieces of a row (of whole 4096-logit groups, whatever the type): one from a row per SM on, below that as many as fill the
// machine once (151936 fp32 logits with 5 alternatives, 500 rows: one piece 52 us, three 63; 250 rows: one 30, two 34; 100
// rows: six 20 us, seven 23; 64 rows: nine 17, ten 18).
int pieces_of(int rows, int vocab, int* piece) {
  const int groups = (vocab + kGroup - 1) / kGroup;
  int n = rows >= kSMs ? 1 : 4 * kSMs / rows;
  n = n < groups ? n : groups;
  n = n < kMaxPieces ? n : kMaxPieces;
  if (n * kMaxGroups < groups) n = (groups + kMaxGroups - 1) / kMaxGroups;      // (at most 16)
  const int per = (groups + n - 1) / n;
  *piece = per * kGroup;
  return (groups + per - 1) / per;
}

constexpr size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

template <typename T>
cudaError_t launch_typed(const LogprobsParams& p, cudaStream_t st) {
  const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && (p.num_rows == 1 || p.row_stride * sizeof(T) % 16 == 0);
  const dim3 grid((unsigned)(p.num_rows * p.pieces));
  auto kernel = p.top > 0 ? (vec ? logprobs_piece_kernel<T, true, true> : logprobs_piece_kernel<T, true, false>)
                          : (vec ? logprobs_piece_kernel<T, false, true> : logprobs_piece_kernel<T, false, false>);
  const cudaError_t e = launch_pdl(kernel, grid, dim3(kLpThreads), 0, st, p);
  if (e != cudaSuccess || p.pieces == 1) return e;
  return launch_pdl(logprobs_join_kernel<T>, dim3(p.num_rows), dim3(kLpThreads), 0, st, p);
}

}  // namespace

size_t logprobs_workspace(int num_rows, int vocab, int top) {
  int piece;
  const size_t pieces = (size_t)pieces_of(num_rows < 1 ? 1 : num_rows, vocab, &piece);
  if (pieces == 1 || num_rows < 1) return 0;
  return align_up(pieces * num_rows * sizeof(float4)) + pieces * num_rows * (size_t)top * sizeof(Key);
}

cudaError_t launch_logprobs(LogprobsParams p, void* workspace, cudaStream_t st) {
  if (p.num_rows == 0) return cudaSuccess;
  p.pieces = pieces_of(p.num_rows, p.vocab, &p.piece);
  p.stats = static_cast<float4*>(workspace);
  p.keys = reinterpret_cast<Key*>(static_cast<char*>(workspace) + align_up((size_t)p.pieces * p.num_rows * sizeof(float4)));
  return p.dtype == SD_LOGITS_F32    ? launch_typed<float>(p, st)
         : p.dtype == SD_LOGITS_BF16 ? launch_typed<__nv_bfloat16>(p, st)
                                     : launch_typed<__half>(p, st);
}

}  // namespace sdv
