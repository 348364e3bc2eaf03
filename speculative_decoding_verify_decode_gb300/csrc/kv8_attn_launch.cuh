// Launch of the block-scaled cache's attention for one (head dim, options)
// kind; each kind is a translation unit of its own, so that they compile side
// by side.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"

namespace sdv {

struct Kv8Plan {
  int hpc, hparts;   // query heads of a KV group per CTA, and CTA parts per group
  int nq, hc;        // query columns, and 16-column chunks of a column half
};
Kv8Plan kv8_plan(int group, int max_nodes, bool mod);

cudaError_t launch_kv8_256(const CUtensorMap&, const CUtensorMap&, const Kv8AttnParams&, const BatchDesc&, int, cudaStream_t);
cudaError_t launch_kv8_128(const CUtensorMap&, const CUtensorMap&, const Kv8AttnParams&, const BatchDesc&, int, cudaStream_t);
cudaError_t launch_kv8_256_mod(const CUtensorMap&, const CUtensorMap&, const Kv8AttnParams&, const BatchDesc&, int, cudaStream_t);
cudaError_t launch_kv8_128_mod(const CUtensorMap&, const CUtensorMap&, const Kv8AttnParams&, const BatchDesc&, int, cudaStream_t);

#ifdef SDV_KV8_DIM
}  // namespace sdv
#include "kv8_attn_kernel.cuh"
namespace sdv {
namespace {

template <int HC>
cudaError_t launch_kv8_hc(const CUtensorMap& mk, const CUtensorMap& mv, const Kv8AttnParams& p, const BatchDesc& bd,
                          cudaStream_t st) {
  constexpr bool kMod = SDV_KV8_MOD != 0;
  constexpr size_t smem = Kv<SDV_KV8_DIM, HC, kMod>::kSmem;
  auto kernel = kv8_attn_kernel<SDV_KV8_DIM, HC, kMod>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<p.grid, kKvThreads, smem, st>>>(mk, mv, p, bd);
  return cudaGetLastError();
}

cudaError_t launch_kv8_kind(const CUtensorMap& mk, const CUtensorMap& mv, const Kv8AttnParams& p, const BatchDesc& bd,
                            int hc, cudaStream_t st) {
  switch (hc) {
    case 1: return launch_kv8_hc<1>(mk, mv, p, bd, st);
    case 2: return launch_kv8_hc<2>(mk, mv, p, bd, st);
    case 3: return launch_kv8_hc<3>(mk, mv, p, bd, st);
    default: return launch_kv8_hc<SDV_KV8_MOD ? 4 : 5>(mk, mv, p, bd, st);
  }
}

}  // namespace
#endif
}  // namespace sdv
