// Host side of the verify attention over the 8-bit block-scaled cache: the
// query-column plan, the page tensor map and the launches.  The kernel is in
// kv8_attn_kernel.cuh, the workspace and the merge of split segments in kv_merge.cuh.
#include <cudaTypedefs.h>

#include "kv8_attn_launch.cuh"
#include "kv_merge.cuh"

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

Layout layout_of(const Kv8Plan& pl, int hkv, int dim, const BatchDesc& bd, int sms) {
  return layout_of(pl.nq, pl.ctas, pl.hparts, hkv, dim, bd, sms);
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
  return p.dim == 256 ? launch_pdl(kv_merge_kernel<256, Kv8AttnParams>, grid, dim3(kMergeThreads), 0, st, p, bd)
                      : launch_pdl(kv_merge_kernel<128, Kv8AttnParams>, grid, dim3(kMergeThreads), 0, st, p, bd);
}

}  // namespace sdv
