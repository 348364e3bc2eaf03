// Host side of the verify attention over the 4-bit cache: the query-column plan
// and the launches.  The kernel is in kv4_attn_kernel.cuh, the workspace and the
// merge of split segments in kv_merge.cuh.
#include "kv4_attn_launch.cuh"
#include "kv_merge.cuh"

namespace sdv {
namespace {

// Query columns of a CTA: as many heads of a KV group as fit, so that the cache is read and widened as few times as
// can be (trees whose 124 to 138 columns fit one part, against two parts of 62 to 72: 23 nodes over 131072 tokens 90 us and
// 114, 31 nodes over 20001 with capped scores 37 and 46).
struct Kv4Plan {
  int hpc, hparts;   // query heads of a KV group per CTA, and CTA parts per group
  int nq;            // query columns of the kernel instance
  int ctas;          // of it per SM
};
Kv4Plan kv4_plan(int group, int max_nodes, int dim) {
  Kv4Plan pl;
  pl.hparts = 1;
  while ((group + pl.hparts - 1) / pl.hparts * max_nodes > 144) ++pl.hparts;
  pl.hpc = (group + pl.hparts - 1) / pl.hparts;
  pl.hparts = (group + pl.hpc - 1) / pl.hpc;
  const int cols = pl.hpc * max_nodes;
  pl.nq = cols <= 16 ? 16 : cols <= 48 ? 48 : cols <= 96 ? 96 : 144;
  pl.ctas = kv4_ctas(pl.nq, dim);
  return pl;
}

}  // namespace

size_t kv4_attn_workspace(int hq, int hkv, int dim, const BatchDesc& bd) {
  const Kv4Plan pl = kv4_plan(hq / hkv, bd.max_nodes, dim);
  return layout_of(pl.nq, pl.ctas, pl.hparts, hkv, dim, bd, sm_count()).total;
}

cudaError_t launch_kv4_attn(Kv4AttnParams p, const BatchDesc& bd, cudaStream_t st) {
  const bool mod = p.softcap > 0.f || p.slopes != nullptr;
  const Kv4Plan pl = kv4_plan(p.group, bd.max_nodes, p.dim);
  p.hpc = pl.hpc;
  p.hparts = pl.hparts;
  p.nq = pl.nq;
  const int sms = sm_count();
  p.grid = sms * pl.ctas;
  const Layout l = layout_of(pl.nq, pl.ctas, pl.hparts, p.hkv, p.dim, bd, sms);
  char* ws = static_cast<char*>(p.workspace);
  p.cum = reinterpret_cast<int*>(ws);
  p.o_part = reinterpret_cast<float*>(ws + l.o);
  p.lse_part = reinterpret_cast<float*>(ws + l.lse);
  const cudaError_t e = p.dim == 256 ? (mod ? launch_kv4_256_mod(p, bd, st) : launch_kv4_256(p, bd, st))
                                     : (mod ? launch_kv4_128_mod(p, bd, st) : launch_kv4_128(p, bd, st));
  if (e != cudaSuccess) return e;
  const dim3 grid(bd.total_nodes, p.hq);
  return p.dim == 256 ? launch_pdl(kv_merge_kernel<256, Kv4AttnParams>, grid, dim3(kMergeThreads), 0, st, p, bd)
                      : launch_pdl(kv_merge_kernel<128, Kv4AttnParams>, grid, dim3(kMergeThreads), 0, st, p, bd);
}

}  // namespace sdv
