// sample_api.cu - the C ABI of sampling and unmasking (include/bdlm.h):
// host-side validation and launches, as in cache_api.cu.
#include <cstdint>

#include "bdlm.h"
#include "cache.cuh"
#include "sample.cuh"

using namespace bdlm;

namespace {

constexpr long long kMaxRows = 1LL << 26;  // eight CTAs of each are a grid
constexpr int kMaxSeqs = 1 << 16;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool good_ptr(const void* p, uintptr_t a) { return p && aligned(p, a); }
bool overlap(const void* x, size_t nx, const void* y, size_t ny) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return x && y && a < b + ny && b < a + nx;
}

}  // namespace

extern "C" {

int bdlm_sample(const void* logits, int32_t dtype, int64_t rows, int32_t vocab, int64_t row_stride, const float* u,
                const bdlm_sampling* how, const int32_t* tokens, int32_t mask_id, int32_t* token, float* logprob,
                bdlm_stream_t stream) {
    set_last_launches(0);
    if (dtype != BDLM_BF16 && dtype != BDLM_F32 && dtype != BDLM_F16) return BDLM_ERR_INVALID_ARG;
    const size_t size = dtype == BDLM_F32 ? 4 : 2;
    if (!good_ptr(logits, size) || !good_ptr(u, 4) || !aligned(tokens, 4) || !good_ptr(token, 4) || !good_ptr(logprob, 4) || !how)
        return BDLM_ERR_INVALID_ARG;
    if ((how->flags & ~BDLM_SAMPLE_NO_MASK) || how->reserved) return BDLM_ERR_INVALID_ARG;
    if (!aligned(how->temperature, 4) || !aligned(how->top_k, 4) || !aligned(how->top_p, 4) || !aligned(how->min_p, 4))
        return BDLM_ERR_INVALID_ARG;
    if (rows < 1 || rows > kMaxRows || vocab < 1 || row_stride < vocab || row_stride > (1LL << 40)) return BDLM_ERR_INVALID_ARG;
    if (vocab > sample::kMaxVocab) return BDLM_ERR_UNSUPPORTED;
    const size_t n = (size_t)rows, logits_bytes = ((n - 1) * (size_t)row_stride + vocab) * size;
    const void* in[] = {u, how->temperature, how->top_k, how->top_p, how->min_p, tokens};
    for (const void* p : in)
        if ((p != tokens && overlap(token, 4 * n, p, 4 * n)) || (p == tokens && p != token && overlap(token, 4 * n, p, 4 * n)) ||
            overlap(logprob, 4 * n, p, 4 * n))
            return BDLM_ERR_INVALID_ARG;
    if (overlap(token, 4 * n, logprob, 4 * n) || overlap(token, 4 * n, logits, logits_bytes) ||
        overlap(logprob, 4 * n, logits, logits_bytes))
        return BDLM_ERR_INVALID_ARG;
    SampleArgs a{};
    a.x = logits;
    a.stride = row_stride;
    a.rows = (int)rows;
    a.vocab = vocab;
    a.u = u;
    a.temperature = how->temperature;
    a.top_k = how->top_k;
    a.top_p = how->top_p;
    a.min_p = how->min_p;
    a.temperature_all = how->temperature_all;
    a.top_k_all = how->top_k_all;
    a.top_p_all = how->top_p_all;
    a.min_p_all = how->min_p_all;
    a.now = tokens;
    a.want = mask_id;
    a.barred = (how->flags & BDLM_SAMPLE_NO_MASK) && mask_id >= 0 && mask_id < vocab ? mask_id : -1;
    a.token = token;
    a.logprob = logprob;
    const int sms = device_sms();
    int launches = 0;
    if (sms <= 0 || launch_sample(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream), &launches) != cudaSuccess)
        return BDLM_ERR_CUDA;
    set_last_launches(launches);
    return BDLM_OK;
}

size_t bdlm_unmask_workspace_bytes(void) { return sizeof(WsHeader); }

int bdlm_unmask(const int32_t* tokens, const int32_t* sampled, const float* logprob, int64_t total_rows,
                const int32_t* cu_rows, int32_t n_seqs, int32_t mask_id, const int32_t* n_min, int32_t n_min_all,
                const float* threshold, float threshold_all, int32_t* out, int32_t* left, void* workspace,
                size_t workspace_bytes, bdlm_stream_t stream) {
    set_last_launches(0);
    if (!good_ptr(tokens, 4) || !good_ptr(sampled, 4) || !good_ptr(logprob, 4) || !good_ptr(cu_rows, 4) || !aligned(n_min, 4) ||
        !aligned(threshold, 4) || !good_ptr(out, 4) || !good_ptr(left, 4))
        return BDLM_ERR_INVALID_ARG;
    if (total_rows < 1 || total_rows > (1LL << 30) || n_seqs < 1 || n_seqs > kMaxSeqs) return BDLM_ERR_INVALID_ARG;
    const size_t n = 4 * (size_t)total_rows, m = 4 * (size_t)n_seqs;
    if ((out != tokens && overlap(out, n, tokens, n)) || overlap(out, n, sampled, n) || overlap(out, n, logprob, n) ||
        overlap(out, n, cu_rows, m + 4) || overlap(out, n, n_min, m) || overlap(out, n, threshold, m) || overlap(out, n, left, m) ||
        overlap(left, m, tokens, n) || overlap(left, m, sampled, n) || overlap(left, m, logprob, n) ||
        overlap(left, m, cu_rows, m + 4) || overlap(left, m, n_min, m) || overlap(left, m, threshold, m))
        return BDLM_ERR_INVALID_ARG;
    if (workspace && (!aligned(workspace, 256) || workspace_bytes < sizeof(WsHeader))) return BDLM_ERR_WORKSPACE;
    UnmaskArgs a{};
    a.now = tokens;
    a.sampled = sampled;
    a.logprob = logprob;
    a.cu_rows = cu_rows;
    a.n_seqs = n_seqs;
    a.total_rows = (int)total_rows;
    a.mask_id = mask_id;
    a.n_min = n_min;
    a.n_min_all = n_min_all;
    a.threshold = threshold;
    a.threshold_all = threshold_all;
    a.out = out;
    a.left = left;
    a.hdr = static_cast<WsHeader*>(workspace);
    int launches = 0;
    if (launch_unmask(a, reinterpret_cast<cudaStream_t>(stream), &launches) != cudaSuccess) return BDLM_ERR_CUDA;
    set_last_launches(launches);
    return BDLM_OK;
}

}  // extern "C"
