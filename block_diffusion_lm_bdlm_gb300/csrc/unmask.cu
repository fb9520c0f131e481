// unmask.cu - which rows of every block keep the tokens that were sampled for
// them in this denoising step.
//
// Of a sequence's rows that are still masked and have a token, those are kept
// whose log-probability is at least the threshold, and if they are fewer than
// n_min the n_min of the largest log-probabilities, of equal ones the first.
// The last one's key is found bit by bit from the highest: a bit stays set if
// n_min keys are at least as large. One CTA per sequence; bound by latency (of
// the loads, and of 32 counts by the CTA where n_min decides): 16 sequences of 32
// rows take 6.8 us, 700 of up to 1024 take 11.
#include "sample.cuh"

namespace bdlm {
namespace {

using sample::order_key;

constexpr int kThreads = 256;
constexpr int kHeld = 4;  // keys that a thread holds in registers; rows beyond 1024 are read again for every count

__global__ void __launch_bounds__(kThreads) unmask_kernel(const UnmaskArgs a) {
    __shared__ int s_n[kThreads / 32];
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto fine = [&](int i, int& lo, int& hi) {
        lo = __ldg(a.cu_rows + i);
        hi = __ldg(a.cu_rows + i + 1);
        return lo >= 0 && hi >= lo && hi <= a.total_rows && (i > 0 || lo == 0);
    };
    auto sum = [&](int x) {  // over the CTA
        x = (int)__reduce_add_sync(0xffffffffu, (unsigned)x);
        __syncthreads();
        if (lane == 0) s_n[warp] = x;
        __syncthreads();
        int y = 0;
        for (int w = 0; w < kThreads / 32; ++w) y += s_n[w];
        return y;
    };
    int lo, hi;
    if (s == 0 && a.hdr) {  // the first CTA looks all offsets over
        int bad = 0x7fffffff;
        for (int i = tid; i < a.n_seqs; i += kThreads)
            if (!fine(i, lo, hi)) bad = min(bad, i);
        bad = __reduce_min_sync(0xffffffffu, bad);
        if (lane == 0) s_n[warp] = bad;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kThreads / 32; ++w) bad = min(bad, s_n[w]);
            a.hdr->error = bad == 0x7fffffff ? 0 : DEV_CHECK;
            a.hdr->info = bad == 0x7fffffff ? 0 : bad;
        }
    }
    if (!fine(s, lo, hi)) return;
    const int rows = hi - lo, most = a.n_min ? __ldg(a.n_min + s) : a.n_min_all;
    const float threshold = a.threshold ? __ldg(a.threshold + s) : a.threshold_all;
    // 0: keeps its token; else the order of its log-probability. NaN comes below everything.
    auto key_at = [&](int i) -> uint32_t {
        if (i >= rows || __ldg(a.now + lo + i) != a.mask_id) return 0u;
        const int drawn = __ldg(a.sampled + lo + i);
        if (drawn < 0 || drawn == a.mask_id) return 0u;  // (a row that was given the mask would still be masked)
        const float x = __ldg(a.logprob + lo + i);
        return x != x ? 1u : order_key(__float_as_uint(x));
    };
    const uint32_t floor = threshold != threshold ? 0xffffffffu : order_key(__float_as_uint(threshold));
    const bool held = rows <= kThreads * kHeld;
    uint32_t k[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) k[j] = held ? key_at(tid + j * kThreads) : 0u;
    auto count = [&](uint32_t least) {  // keys from `least` on
        int n = 0;
        if (held) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j) n += k[j] >= least;
        } else {
            for (int i = tid; i < rows; i += kThreads) n += key_at(i) >= least;
        }
        return sum(n);
    };
    const int sure = count(max(floor, 2u)), can = count(1u);
    uint32_t cut = max(floor, 2u);  // keys from here on are kept, and of those just below it ...
    int ties = 0;                   // ... the first `ties`
    if (sure < most) {
        if (can <= most) {
            cut = 1u;
        } else {
            uint32_t key = 0;
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t next = key | 1u << bit;
                if (count(next) >= most) key = next;
            }
            const int above = key == 0xffffffffu ? 0 : count(key + 1);
            cut = key + 1;  // (no key is 2^32 - 1: that would be a NaN)
            ties = most - above;
        }
    }
    int masked = 0, kept = 0, seen = 0;  // seen: rows of the tied key before this stretch
    for (int i0 = 0; i0 < rows; i0 += kThreads) {
        const int i = i0 + tid;
        const uint32_t key = key_at(i);
        bool keep = key >= cut;
        if (ties > 0) {
            const bool tied = key == cut - 1;
            const unsigned who = __ballot_sync(0xffffffffu, tied);
            __syncthreads();
            if (lane == 0) s_n[warp] = __popc(who);
            __syncthreads();
            int before = seen;
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) before += s_n[w];
                seen += s_n[w];
            }
            keep = keep || (tied && before + __popc(who & ((1u << lane) - 1)) < ties);
        }
        if (i < rows) {
            const int now = __ldg(a.now + lo + i);
            masked += now == a.mask_id;
            kept += keep;
            const int next = keep ? __ldg(a.sampled + lo + i) : now;
            if (a.out != a.now || keep) a.out[lo + i] = next;
        }
    }
    const int left = sum(masked - kept);
    if (tid == 0) a.left[s] = left;
}

}  // namespace

cudaError_t launch_unmask(const UnmaskArgs& a, cudaStream_t st, int* launches) {
    unmask_kernel<<<a.n_seqs, kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace bdlm
