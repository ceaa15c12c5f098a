// The tcgen05 attention of dflash_kv4_prefix_attention: the groups' rows over their prefixes, and blocks
// of many rows over their own cells.
#include "kv4_attention_tc.cuh"

namespace dflash {

cudaError_t launch_kv4_attn_tc_prefix(int d, const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st) {
  return launch_d<kKv4Prefix>(d, a, most, jobs, st);
}
cudaError_t launch_kv4_attn_tc_own(int d, const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st) {
  return launch_d<kKv4Own>(d, a, most, jobs, st);
}

}  // namespace dflash
