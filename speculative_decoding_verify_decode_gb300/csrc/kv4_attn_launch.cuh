// Launch of the 4-bit cache's attention for one (head dim, options) kind; each
// kind is a translation unit of its own, so that they compile side by side.
#pragma once

#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace sdv {

cudaError_t launch_kv4_256(const Kv4AttnParams&, const BatchDesc&, cudaStream_t);
cudaError_t launch_kv4_128(const Kv4AttnParams&, const BatchDesc&, cudaStream_t);
cudaError_t launch_kv4_256_mod(const Kv4AttnParams&, const BatchDesc&, cudaStream_t);
cudaError_t launch_kv4_128_mod(const Kv4AttnParams&, const BatchDesc&, cudaStream_t);

#ifdef SDV_KV4_DIM
}  // namespace sdv
#include "kv4_attn_kernel.cuh"
namespace sdv {
namespace {

template <int NG, int CC>
cudaError_t launch_kv4_cols(const Kv4AttnParams& p, const BatchDesc& bd, cudaStream_t st) {
  using K = Kv4<SDV_KV4_DIM, NG, CC, SDV_KV4_MOD != 0>;
  const auto kernel = kv4_attn_kernel<SDV_KV4_DIM, NG, CC, SDV_KV4_MOD != 0>;
  // The roles share out the registers of the launch: with fewer than these they would wait for one another.
  static std::atomic<int> regs{0};
  if (regs.load() == 0) {
    cudaFuncAttributes a;
    const cudaError_t asked = cudaFuncGetAttributes(&a, kernel);
    if (asked != cudaSuccess) return asked;
    regs.store(a.numRegs);
  }
  if (regs.load() < K::kLaunchRegs) return cudaErrorLaunchOutOfResources;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(p.grid), dim3(K::kThreads), K::kSmem, st, p, bd);
}

cudaError_t launch_kv4_kind(const Kv4AttnParams& p, const BatchDesc& bd, cudaStream_t st) {
  switch (p.nq) {
    case 16: return launch_kv4_cols<1, 1>(p, bd, st);
    case 48: return launch_kv4_cols<1, 3>(p, bd, st);
    case 96: return launch_kv4_cols<2, 3>(p, bd, st);
    case 144: return launch_kv4_cols<3, 3>(p, bd, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
#endif
}  // namespace sdv
