// cache_attn_runs_d64.cu - the attention kernel over shared and own pages for head dimension 64.
#include "cache_attn_tc.cuh"

namespace bdlm {
cudaError_t launch_cache_attn_runs_d64(const CacheAttnArgs& a, int ctas, cudaStream_t st) { return cattn::launch_d<64, true>(a, ctas, st); }
}  // namespace bdlm
