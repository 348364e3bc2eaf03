// Instances of the block-scaled cache's attention: head dim 256, capped scores or a distance bias.
#define SDV_KV8_DIM 256
#define SDV_KV8_MOD 1
#include "kv8_attn_launch.cuh"

namespace sdv {

cudaError_t launch_kv8_256_mod(const CUtensorMap& mk, const CUtensorMap& mv, const Kv8AttnParams& p, const BatchDesc& bd,
                           cudaStream_t st) {
  return launch_kv8_kind(mk, mv, p, bd, st);
}

}  // namespace sdv
