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
  int nq;            // query columns of the kernel instance
  int ctas;          // of it per SM
};
Kv8Plan kv8_plan(int group, int max_nodes, int dim, bool mod, int kv_rows);   // kv_rows: sequences x KV heads

cudaError_t launch_kv8_256(const CUtensorMap&, const CUtensorMap&, const Kv8AttnParams&, const BatchDesc&, cudaStream_t);
cudaError_t launch_kv8_128(const CUtensorMap&, const CUtensorMap&, const Kv8AttnParams&, const BatchDesc&, cudaStream_t);
cudaError_t launch_kv8_256_mod(const CUtensorMap&, const CUtensorMap&, const Kv8AttnParams&, const BatchDesc&, cudaStream_t);
cudaError_t launch_kv8_128_mod(const CUtensorMap&, const CUtensorMap&, const Kv8AttnParams&, const BatchDesc&, cudaStream_t);

#ifdef SDV_KV8_DIM
}  // namespace sdv
#include "kv8_attn_kernel.cuh"
namespace sdv {
namespace {

template <int NG, int CC>
cudaError_t launch_kv8_cols(const CUtensorMap& mk, const CUtensorMap& mv, const Kv8AttnParams& p, const BatchDesc& bd,
                            cudaStream_t st) {
  using K = Kv<SDV_KV8_DIM, NG, CC, SDV_KV8_MOD != 0>;
  auto kernel = kv8_attn_kernel<SDV_KV8_DIM, NG, CC, SDV_KV8_MOD != 0>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(p.grid), dim3(K::kThreads), K::kSmem, st, mk, mv, p, bd);
}

cudaError_t launch_kv8_kind(const CUtensorMap& mk, const CUtensorMap& mv, const Kv8AttnParams& p, const BatchDesc& bd,
                            cudaStream_t st) {
  switch (p.nq) {
    case 16: return launch_kv8_cols<1, 1>(mk, mv, p, bd, st);
#if SDV_KV8_DIM == 128                     // see kv8_plan
    case 32: return launch_kv8_cols<1, 2>(mk, mv, p, bd, st);
#endif
    case 48: return launch_kv8_cols<3, 1>(mk, mv, p, bd, st);
    case 96: return launch_kv8_cols<3, 2>(mk, mv, p, bd, st);
#if !(SDV_KV8_MOD && SDV_KV8_DIM == 256)
    case 144: return launch_kv8_cols<3, 3>(mk, mv, p, bd, st);
#endif
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
#endif
}  // namespace sdv
