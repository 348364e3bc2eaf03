// Instances of the 4-bit cache's attention: head dim 128, plain scores.
#define SDV_KV4_DIM 128
#define SDV_KV4_MOD 0
#include "kv4_attn_launch.cuh"

namespace sdv {

cudaError_t launch_kv4_128(const Kv4AttnParams& p, const BatchDesc& bd, cudaStream_t st) {
  return launch_kv4_kind(p, bd, st);
}

}  // namespace sdv
