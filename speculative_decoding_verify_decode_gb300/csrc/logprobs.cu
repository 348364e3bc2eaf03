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
// Top.  A logit and its index make one 64-bit key that orders as they do (value, then
// the smaller index), so ties need no care and the `top` largest keys are one set.  A
// CTA keeps them in a list with a bar, the smallest key that can still matter; a tile's
// keys above the bar join the list, which is cut back to the `top` largest when it has
// grown.  Before there is a bar one is taken from the tile: in each warp the j-th
// largest of the threads' maxima with j = ceil(top / warps), the smallest of
// them over the warps; at least `top` keys are no smaller.  Whatever the data,
// the list has room for all of a tile (sorted rows are slow, not wrong).
//
// Bound by HBM for many rows: 6 instructions and one ex2 a logit.  Rows are
// cut into pieces over CTAs where there are few, and joined by a second launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace sdv {
namespace {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kPer = 16;                        // logits of a thread that are looked at together
constexpr int kGroup = kLpThreads * kPer;
constexpr int kListCut = 64;                    // the list is cut back when it is longer
constexpr int kFew = 2 * kLpThreads;            // keys that are ranked one by one
constexpr int kListMax = kListCut + kGroup;
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
  __device__ __forceinline__ void join(Stats o, float f) {
    if (o.m > m) rise(o.m, f);
    if (m > o.m) o.rise(m, f);
    c += o.c;
    s += o.s;
    w += o.w;
  }
};

struct LpShared {
  Key list[kListMax];
  Key bar;
  int n;             // keys in the list
  int count;         // of a search
  Key few[kFew];     // what a cut looks at
  uint32_t warp_bar[kLpWarps];
  Key top_of[kLpWarps];
  float m[kLpWarps], c[kLpWarps], s[kLpWarps], w[kLpWarps];
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

// A 16-byte piece as floats.
template <typename T>
struct Load;
template <>
struct Load<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ void put(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
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
};
template <>
struct Load<__half> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void put(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
template <typename T>
__device__ __forceinline__ float value_of(T x) { return static_cast<float>(x); }

// The logit of a row's t-th given token (one a thread); -infinity where it is none.
static_assert(SD_LOGPROBS_MAX_GIVEN <= kLpThreads, "a thread for each given token");
template <typename T>
__device__ __forceinline__ float given_logit(const LogprobsParams& p, int row) {
  if ((int)threadIdx.x >= p.given) return -INFINITY;
  const int v = p.tokens[(size_t)row * p.given + threadIdx.x];
  return v >= 0 && v < p.vocab ? value_of(static_cast<const T*>(p.logits)[(long long)row * p.row_stride + v]) : -INFINITY;
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
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    Stats o;
    o.m = __shfl_xor_sync(0xffffffffu, st.m, d);
    o.c = __shfl_xor_sync(0xffffffffu, st.c, d);
    o.s = __shfl_xor_sync(0xffffffffu, st.s, d);
    o.w = __shfl_xor_sync(0xffffffffu, st.w, d);
    // the lower lane's first, so that both lanes compute the same
    Stats a = (lane & d) ? o : st;
    a.join((lane & d) ? st : o, f);
    st = a;
  }
  if (lane == 0) { sh.m[warp] = st.m; sh.c[warp] = st.c; sh.s[warp] = st.s; sh.w[warp] = st.w; }
  __syncthreads();
  st.m = sh.m[0]; st.c = sh.c[0]; st.s = sh.s[0]; st.w = sh.w[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) {
    Stats o;
    o.m = sh.m[w]; o.c = sh.c[w]; o.s = sh.s[w]; o.w = sh.w[w];
    st.join(o, f);
  }
  return st;
}

// VEC: the rows start on 16 bytes and so does every 16-byte piece of them.
template <typename T, bool TOP, bool VEC>
__global__ void __launch_bounds__(kLpThreads, TOP ? 4 : 5) logprobs_piece_kernel(const LogprobsParams p) {
  __shared__ LpShared sh;
  constexpr int kVec = Load<T>::kVec, kTile = kLpTile<T>, kPieces = kPer / kVec, kGroups = kTile / kGroup;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int row = blockIdx.x / p.pieces, piece = blockIdx.x - row * p.pieces;
  const T* x = static_cast<const T*>(p.logits) + (long long)row * p.row_stride;
  const int begin = piece * p.piece, end = min(p.vocab, begin + p.piece);
  const float f = p.inv_t * kLog2eLp;
  pdl_wait();
  if (TOP && t == 0) { sh.n = 0; sh.bar = 0; }
  Stats st;
  st.m = -INFINITY;
  st.c = st.s = st.w = 0.f;
  bool bad = false;
  // A thread's logits of a tile: 16-byte piece j at begin + (j * kLpThreads + t) * kVec.
  uint4 raw[4];
  auto fetch = [&](int at) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = at + (j * kLpThreads + t) * kVec;
      if (VEC && v + kVec <= end) {
        raw[j] = __ldcs(reinterpret_cast<const uint4*>(x + v));
      } else {
        // what lies past the end counts as tokens that cannot come
        alignas(16) T e[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) e[k] = v + k < end ? x[v + k] : static_cast<T>(-INFINITY);
        raw[j] = *reinterpret_cast<const uint4*>(e);
      }
    }
  };
  fetch(begin);
#pragma unroll 1
  for (int tile = begin; tile < end; tile += kTile) {
    uint4 held[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) held[j] = raw[j];
    if (tile + kTile < end) fetch(tile + kTile);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
    const int at = tile + g * kGroup;
    if (at >= end) break;
    float y[kPer];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) Load<T>::put(held[g * kPieces + j], y + j * kVec);
    float top = y[0];
#pragma unroll
    for (int e = 1; e < kPer; ++e) top = max_nan(top, y[e]);
    bad |= top != top;
    const float warp_top = warp_max(top);
    // a logit of -infinity: e^d = 0, and d is kept finite so that the product is 0
    if (warp_top >= st.m) {
      if (warp_top > st.m) st.rise(warp_top, f);
      const float m = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const float d = fmaxf((y[e] - m) * f, -1e30f), a = fast_exp2(d);
        const bool at_top = y[e] == m;
        st.c += at_top ? 1.f : 0.f;
        st.s += at_top ? 0.f : a;
        st.w = fmaf(a, d, st.w);
      }
      bad |= warp_top == INFINITY;
    } else {
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
    if (TOP) {
      if (at == begin) {
        // a first bar (32 bits of it): in each warp the j-th largest of the threads' maxima
        uint32_t o = order_of(top);
        if (top != top) o = 0u;
        const uint32_t jth = warp_jth(o, (p.top + kLpWarps - 1) / kLpWarps);
        if (lane == 0) sh.warp_bar[warp] = jth;
        __syncthreads();
        uint32_t bar = sh.warp_bar[0];
#pragma unroll
        for (int w2 = 1; w2 < kLpWarps; ++w2) bar = min(bar, sh.warp_bar[w2]);
        if (t == 0) sh.bar = (Key)bar << 32;
        __syncthreads();
      }
      const Key bar = sh.bar;
      const float bar_value = order_value((uint32_t)(bar >> 32));   // (NaN for 0: every comparison below then holds)
      // this thread's logits that reach the bar, a bit each: few, taken one after the other
      uint32_t pass = 0;
      bool pushed = false;
      if (__any_sync(0xffffffffu, !(top < bar_value))) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) pass |= y[e] < bar_value ? 0u : 1u << e;
#pragma unroll 1
        while (__any_sync(0xffffffffu, pass != 0)) {
          const int e0 = __ffs(pass) - 1;      // -1: none
          float value = 0.f;
#pragma unroll
          for (int e = 0; e < kPer; ++e) value = e0 == e ? y[e] : value;
          const int v = at + ((e0 / kVec) * kLpThreads + t) * kVec + e0 % kVec;
          const Key k = key_of(value, v);
          const bool ok = pass != 0 && v < end && k >= bar && value == value;
          const uint32_t who = __ballot_sync(0xffffffffu, ok);
          if (who != 0u) {
            int place = 0;
            if (lane == 0) place = atomicAdd(&sh.n, __popc(who));
            place = __shfl_sync(0xffffffffu, place, 0) + __popc(who & ((1u << lane) - 1u));
            if (ok) sh.list[place] = k;
            pushed = true;
          }
          pass &= pass - 1u;
        }
      }
      // a tile in which nobody had anything leaves the list as it was
      if (__syncthreads_or(pushed ? 1 : 0)) {
        const int n = sh.n;
        __syncthreads();
        if (n > kListCut || (at == begin && n > p.top)) {
          cut_list(sh, n, p.top);
          if (t == 0) {
            sh.n = min(n, p.top);
            if (n >= p.top) sh.bar = sh.list[p.top - 1];
          }
          __syncthreads();
        }
      }
    }
    }
  }
  if (TOP) {
    const int n = sh.n;
    __syncthreads();
    cut_list(sh, n, p.top);
    // a piece with fewer than `top` keys (the last of a row, or one with NaN): the rest sort behind everything
    for (int i = min(n, p.top) + t; i < p.top; i += kLpThreads) sh.list[i] = 0;
  }
  const bool any_bad = __syncthreads_or(bad ? 1 : 0) != 0;
  st = block_stats(sh, st, f);
  if (p.pieces == 1) {
    finish_row<T>(p, sh, row, st, any_bad, given_logit<T>(p, row));
  } else {
    if (t == 0) p.stats[blockIdx.x] = make_float4(st.m, any_bad ? NAN : st.c, st.s, st.w);
    if (TOP)
      for (int i = t; i < p.top; i += kLpThreads) p.keys[(size_t)blockIdx.x * p.top + i] = sh.list[i];
  }
}

// The pieces of a row joined: at most kMaxPieces of them.
constexpr int kMaxPieces = 128;
static_assert(kMaxPieces * SD_LOGPROBS_MAX_TOP <= kListMax && kMaxPieces <= kLpThreads, "a row's keys fit the list");

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_join_kernel(const LogprobsParams p) {
  __shared__ LpShared sh;
  const int row = blockIdx.x, t = threadIdx.x;
  const float f = p.inv_t * kLog2eLp;
  pdl_wait();
  const float given = given_logit<T>(p, row);
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
    if ((t & 31) == 0) sh.top_of[t >> 5] = (Key)hi << 32 | lo;
    __syncthreads();
    Key bar = 0;
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) bar = sh.top_of[w] > bar ? sh.top_of[w] : bar;
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

// Pieces of a row (of whole 4096-logit groups, whatever the type): one while the rows make three waves of CTAs, else so
// many that there is about one wave, and none smaller than a group.
int pieces_of(int rows, int vocab, int* piece) {
  const int groups = (vocab + kGroup - 1) / kGroup, wave = 4 * kSMs;
  int n = rows >= 3 * wave ? 1 : rows > wave / 2 ? (2 * wave + rows - 1) / rows : (wave + rows - 1) / rows;
  n = n < groups ? n : groups;
  n = n < kMaxPieces ? n : kMaxPieces;
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
