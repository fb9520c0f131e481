// cache_attn_d128.cu - the attention kernel over the cache for head dimension 128.
#include "cache_attn_tc.cuh"

namespace bdlm {
cudaError_t launch_cache_attn_d128(const CacheAttnArgs& a, int ctas, cudaStream_t st) { return cattn::launch_d<128>(a, ctas, st); }
}  // namespace bdlm
