// Host side of the verify attention over the 8-bit block-scaled cache: the
// query-column plan, the workspace, the page tensor map, the merge of split
// segments, and the launches.  The kernel is in kv8_attn_kernel.cuh.
#include <cudaTypedefs.h>

#include "kv8_attn_launch.cuh"

namespace sdv {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// The codes viewed as 4-D: x = 128 codes of a row, y = slot within an 8-slot half page, z = 128-dim block,
// w = half page of one KV head.  A box of {128, 8, D / 128, 2} is one page of one head, landing as
// [half][block][8 slots][128 B] with the 128-byte swizzle: two 8-row groups of a K tile or a V half tile.
bool page_map(CUtensorMap* map, const void* cache, const Kv8AttnParams& p) {
  auto fn = tensor_map_fn();
  if (fn == nullptr) return false;
  const cuuint32_t blocks = (cuuint32_t)(p.dim / 128);
  cuuint64_t dims[4] = {128, 8, blocks, (cuuint64_t)p.num_pool_pages * p.hkv * 2};
  cuuint64_t strides[3] = {(cuuint64_t)p.dim, 128, (cuuint64_t)p.dim * 8};
  cuuint32_t box[4] = {128, 8, blocks, 2};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(cache), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    cudaGetLastError();   // no device here
    return kSMs;
  }
  return sms;
}

// Log-sum-exp merge of the segments that piece borders cut: o = sum 2^(lse_s - M) o_s / sum 2^(lse_s - M).
// One block per (node row, query head): four warps each take every fourth partial, a lane D / 32 dims, with the
// loads of kBatch partials in flight per warp (40 partials in one round of latency).
constexpr int kMergeThreads = 128, kMergeWarps = 4, kBatch = 10;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) kv8_merge_kernel(const Kv8AttnParams p, const BatchDesc bd) {
  constexpr int E = D / 32;   // dims per lane
  const int r = blockIdx.x, h = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int b = 0, hi = bd.batch - 1;
  while (b < hi) {
    const int mid = (b + hi + 1) >> 1;
    if (bd.q_indptr[mid] <= r) b = mid; else hi = mid - 1;
  }
  const int g = h / p.group, c = (h % p.group) / p.hpc, part0 = c * p.hpc;
  const int hpc = min(p.hpc, p.group - part0);
  const int col = (r - bd.q_indptr[b]) * hpc + h % p.group - part0;
  const int parts = p.hkv * p.hparts, s = g * p.hparts + c;
  int L = p.ctx_lens[b];
  L = L < 0 ? 0 : min(L, p.max_pages * kPage);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the attention kernel's partials and unit sums
  const int per = p.cum[kMaxBatch + 1], extra = p.cum[kMaxBatch + 2];
  const int cum = p.cum[b], line = (p.cum[b + 1] - cum) / parts;
  const int units = extra < 0 ? line : 1 + extra + (L - window_base(L, p.window, kTileTokens) + kTileTokens - 1) / kTileTokens;
  const int u0 = cum + s * line, k0 = u0 / per, n = (u0 + units - 1) / per - k0 + 1;
  if (n == 1) return;   // written directly
  const size_t slot0 = (size_t)k0 + b * parts + s;
  float mx = -INFINITY, den = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int base = warp; base < n; base += kMergeWarps * kBatch) {
    float w[kBatch];
    float o[kBatch][E];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + k * kMergeWarps;
      const size_t at = (slot0 + min(i, n - 1)) * p.nq + col;
      w[k] = i < n ? p.lse_part[at] : -INFINITY;
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(&o[k][e]) = *reinterpret_cast<const float4*>(p.o_part + at * D + lane * E + e);
    }
    float bm = mx;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) bm = fmaxf(bm, w[k]);
    const float a = mx == -INFINITY ? 0.f : fast_exp2(mx - bm);
    den *= a;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= a;
    mx = bm;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (w[k] == -INFINITY) continue;                   // nothing visible there, or padding (a NaN goes on)
      const float f = fast_exp2(w[k] - mx);
      den += f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += f * o[k][e];
    }
  }
  // Every load is under way or done: the next kernel's blocks may come as this one's leave (at the start of the block
  // they took the SMs of a large merge: 512 rows of 16 partials 209 -> 224 us for the whole call).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float s_m[kMergeWarps], s_d[kMergeWarps], s_acc[kMergeWarps][D];
  if (lane == 0) { s_m[warp] = mx; s_d[warp] = den; }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
  __syncthreads();
  float m = s_m[0];
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) m = fmaxf(m, s_m[w]);
  float f[kMergeWarps], d = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    f[w] = s_m[w] == -INFINITY && s_d[w] == 0.f ? 0.f : fast_exp2(s_m[w] - m);
    d += f[w] * s_d[w];
  }
  const float inv = 1.f / d;
  constexpr int T = D / 2;    // threads that write a pair of dims
  if (threadIdx.x < T) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      const float2 v = *reinterpret_cast<const float2*>(&s_acc[w][2 * threadIdx.x]);
      x += f[w] * v.x;
      y += f[w] * v.y;
    }
    *reinterpret_cast<__nv_bfloat162*>(p.out + ((size_t)r * p.hq + h) * D + 2 * threadIdx.x) =
        __floats2bfloat162_rn(x * inv, y * inv);
  }
  if (p.lse != nullptr && threadIdx.x == 0) p.lse[(size_t)r * p.hq + h] = (m + fast_log2(d)) * kLn2;
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct Layout {
  size_t o, lse, total;   // cum at 0
};
Layout layout_of(const Kv8Plan& pl, int hkv, int dim, const BatchDesc& bd, int sms) {
  // a piece and a segment name a partial; along the line of units their numbers rise together
  const size_t slots = (size_t)sms * pl.ctas + (size_t)bd.batch * hkv * pl.hparts;
  Layout l;
  l.o = align_up((kMaxBatch + 3) * sizeof(int));
  l.lse = l.o + align_up(slots * pl.nq * dim * sizeof(float));
  l.total = l.lse + align_up(slots * pl.nq * sizeof(float));
  return l;
}

}  // namespace

// Query columns of a CTA: as many heads of a KV group as fit, so that the cache is read as few times as can be (capped
// or biased scores over 256 dims stop at 96: the wider columns' slopes find no room beside the operands).  Up to 16
// columns, i.e. single tokens, two CTAs of one softmax group share an SM (64 sequences, 1 to 32768 tokens, 128 dims:
// 394 us against 614 for one CTA of three groups; one sequence of 512 tokens 10.9 against 11.3).  So do 17 to 32 columns
// of 128 dims where there are segments enough to fill both (64 sequences of 8 nodes: 213 us against 226; 8 sequences: 37.8
// against 45.5); a few segments take one CTA of three groups, whose single tile is shorter (one sequence of 8 nodes over
// 8192 tokens: 15.1 us against 16.9), and so do 256 dims, where half an SM's shared memory holds one K tile (64 sequences
// of 5 nodes: 147 us against 155).
Kv8Plan kv8_plan(int group, int max_nodes, int dim, bool mod, int kv_rows) {
  const int most = mod && dim == 256 ? 96 : 144;
  Kv8Plan pl;
  pl.hparts = 1;
  while ((group + pl.hparts - 1) / pl.hparts * max_nodes > most) ++pl.hparts;
  pl.hpc = (group + pl.hparts - 1) / pl.hparts;
  pl.hparts = (group + pl.hpc - 1) / pl.hpc;
  const int cols = pl.hpc * max_nodes;
  const bool two = cols <= 16 || (cols <= 32 && dim == 128 && kv_rows * pl.hparts >= 64);
  pl.nq = two ? (cols <= 16 ? 16 : 32) : cols <= 48 ? 48 : cols <= 96 ? 96 : 144;
  pl.ctas = two ? 2 : 1;
  return pl;
}

size_t kv8_attn_workspace(int hq, int hkv, int dim, const BatchDesc& bd) {
  // the query does not know whether scores will be capped or biased
  const int sms = sm_count();
  const size_t a = layout_of(kv8_plan(hq / hkv, bd.max_nodes, dim, false, bd.batch * hkv), hkv, dim, bd, sms).total;
  const size_t b = layout_of(kv8_plan(hq / hkv, bd.max_nodes, dim, true, bd.batch * hkv), hkv, dim, bd, sms).total;
  return a > b ? a : b;
}

cudaError_t launch_kv8_attn(Kv8AttnParams p, const BatchDesc& bd, cudaStream_t st) {
  const bool mod = p.softcap > 0.f || p.slopes != nullptr;
  const Kv8Plan pl = kv8_plan(p.group, bd.max_nodes, p.dim, mod, bd.batch * p.hkv);
  p.hpc = pl.hpc;
  p.hparts = pl.hparts;
  p.nq = pl.nq;
  const int sms = sm_count();
  p.grid = sms * pl.ctas;
  const Layout l = layout_of(pl, p.hkv, p.dim, bd, sms);
  char* ws = static_cast<char*>(p.workspace);
  p.cum = reinterpret_cast<int*>(ws);
  p.o_part = reinterpret_cast<float*>(ws + l.o);
  p.lse_part = reinterpret_cast<float*>(ws + l.lse);
  CUtensorMap mk, mv;
  if (!page_map(&mk, p.k_cache, p) || !page_map(&mv, p.v_cache, p)) return cudaErrorInvalidValue;
  cudaError_t e = p.dim == 256 ? (mod ? launch_kv8_256_mod(mk, mv, p, bd, st) : launch_kv8_256(mk, mv, p, bd, st))
                               : (mod ? launch_kv8_128_mod(mk, mv, p, bd, st) : launch_kv8_128(mk, mv, p, bd, st));
  if (e != cudaSuccess) return e;
  const dim3 grid(bd.total_nodes, p.hq);
  return p.dim == 256 ? launch_pdl(kv8_merge_kernel<256>, grid, dim3(kMergeThreads), 0, st, p, bd)
                      : launch_pdl(kv8_merge_kernel<128>, grid, dim3(kMergeThreads), 0, st, p, bd);
}

}  // namespace sdv
