// Instances of the block-scaled cache's attention: head dim 128, plain scores.
#define SDV_KV8_DIM 128
#define SDV_KV8_MOD 0
#include "kv8_attn_launch.cuh"

namespace sdv {

cudaError_t launch_kv8_128(const CUtensorMap& mk, const CUtensorMap& mv, const Kv8AttnParams& p, const BatchDesc& bd,
                           cudaStream_t st) {
  return launch_kv8_kind(mk, mv, p, bd, st);
}

}  // namespace sdv
