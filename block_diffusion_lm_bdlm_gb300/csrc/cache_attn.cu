// cache_attn.cu - launches the attention over the paged cache and the join of
// its partial results.
#include "cache_merge.cuh"

namespace bdlm {

size_t cache_attn_scratch_bytes(long long total_rows, int H, int Hk, int D, int) {
    const int rows = slot_rows(total_rows, H / Hk);
    return sizeof(ShareRec) * kMaxCtas + sizeof(float) * 2 * kMaxCtas * (size_t)slot_floats(rows, D);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int num_sms, cudaStream_t st, int* launches) {
    const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    cudaError_t e = a.c.D == 128 ? launch_cache_attn_d128(a, ctas, st) : launch_cache_attn_d64(a, ctas, st);
    if (e == cudaSuccess) e = launch_merge<false>(a, ctas, st);
    if (e == cudaSuccess) *launches += 2;
    return e;
}

}  // namespace bdlm
