// The tcgen05 attention of dflash_kv4_attention.
#include "kv4_attention_tc.cuh"

namespace dflash {

cudaError_t launch_kv4_attn_tc(int d, const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st) {
  return launch_d<kKv4Plain>(d, a, most, jobs, st);
}

}  // namespace dflash
