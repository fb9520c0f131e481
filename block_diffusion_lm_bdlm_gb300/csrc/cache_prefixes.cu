// cache_prefixes.cu - which neighbouring sequences of a call read which pages
// together.
//
// Mathematics. Of the sequences that have rows, in order, c_i is the number of
// pages that the i-th and the next begin with alike, counting pages that lie
// wholly below the rows of both. A run of sequences shares the least c between
// its members and saves (members - 1) times that many page reads. The cut into
// runs that saves most in all is found from left to right: with best[j] for
// the first j sequences,
//   best[j] = max over i of best[i] + (j - i - 1) min(c_i .. c_{j-2}),
// over runs of at most kLongest sequences; of cuts as good, the one with the
// shortest last run.
//
// Bound. Both kernels are bound by latency. The first has a warp per sequence
// and compares 256 table entries at a time; the second's recurrence is a chain
// of one step per sequence, which one warp does with eight starts per lane: 64
// sequences take 10.2 us in all, 600 take 48, about 140 clocks a step. (With the
// distance found by a second reduction they took 14 and 67.)
#include "cache.cuh"

namespace bdlm {
namespace {

constexpr int kLongest = 256;
static_assert(kLongest == 8 * 32, "a warp has eight starts per lane");
constexpr int kThreads = 256;
constexpr int kMost = 32767;  // pages that count, so that 256 times what a run saves stays in 32 bits
constexpr int kNoRows = -1, kMalformed = -2;

// Pages of sequence r that lie wholly below its rows.
__device__ __forceinline__ int covered(const CacheView& c, const SeqRows& r) {
    return max(0, min(r.len, r.pos0)) >> c.page_shift;
}

// alike[s]: pages that sequence s and the next one with rows begin with alike; kNoRows; kMalformed.
__global__ void __launch_bounds__(kThreads) alike_kernel(const CachePrefixArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, s = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), n = a.c.n_seqs;
    if (s >= n) return;
    const SeqRows r = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s);
    int got = !r.ok ? kMalformed : r.rows == 0 ? kNoRows : 0;
    if (got == 0) {
        int next = -1;  // the next sequence with rows
        for (int j0 = s + 1; j0 < n && next < 0; j0 += 32) {
            const int j = j0 + lane;
            const unsigned hit = __ballot_sync(0xffffffffu, j < n && __ldg(a.cu_rows + j + 1) > __ldg(a.cu_rows + j));
            if (hit) next = j0 + __ffs(hit) - 1;
        }
        if (next >= 0) {
            const SeqRows q = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, next);
            const int most = q.ok ? min(min(covered(a.c, r), covered(a.c, q)), kMost) : 0;
            const int* x = a.c.table + (long long)s * a.c.max_pages;
            const int* y = a.c.table + (long long)next * a.c.max_pages;
            got = most;
            for (int at = 0; at < most; at += 256) {
                int p[8], q8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int i = at + 32 * k + lane;
                    p[k] = i < most ? __ldg(x + i) : 0;
                    q8[k] = i < most ? __ldg(y + i) : 0;
                }
                int first = -1;
#pragma unroll
                for (int k = 7; k >= 0; --k) {
                    const unsigned off = __ballot_sync(0xffffffffu, p[k] != q8[k]);
                    if (off) first = at + 32 * k + __ffs(off) - 1;
                }
                if (first >= 0) {
                    got = first;
                    break;
                }
            }
        }
    }
    if (lane == 0) a.scratch[s] = got;
}

// Shared memory: of the sequences with rows their numbers and c, how far back the last run of the best cut of those up to
// each begins, and the starts of the runs.
size_t cut_smem(int n) { return (size_t)n * (4 + 4 + 4 + 1) + 16; }

__global__ void __launch_bounds__(kThreads) cut_kernel(const CachePrefixArgs a) {
    extern __shared__ int sm[];
    const int n = a.c.n_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* busy = sm;
    int* c = busy + n;
    int* starts = c + n;
    uint8_t* back = reinterpret_cast<uint8_t*>(starts + n);
    __shared__ int s_warp[kThreads / 32], s_runs, s_bad;
    int *first = a.runs, *end = a.runs + n, *shared = a.runs + 2 * (long long)n;
    if (tid == 0) s_bad = 0x7fffffff;
    for (int s = tid; s < n; s += kThreads) {
        first[s] = s;
        end[s] = s + 1;
        shared[s] = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    int m = 0;
    for (int s0 = 0; s0 < n; s0 += kThreads) {
        const int s = s0 + tid, x = s < n ? __ldcg(a.scratch + s) : kNoRows;
        if (x == kMalformed) atomicMin(&s_bad, s);
        const unsigned has = __ballot_sync(0xffffffffu, x >= 0);
        if (lane == 0) s_warp[warp] = __popc(has);
        __syncthreads();
        int before = m;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            m += s_warp[w];
        }
        if (x >= 0) {
            const int at = before + __popc(has & ((1u << lane) - 1));
            busy[at] = s;
            c[at] = x;
        }
        __syncthreads();
    }
    if (tid == 0) {
        a.hdr->error = s_bad == 0x7fffffff ? 0 : DEV_CHECK;
        a.hdr->info = s_bad == 0x7fffffff ? 0 : s_bad;
    }
    if (s_bad != 0x7fffffff) return;  // nothing is shared then
    if (warp == 0) {
        // Start i lies in lane i % 32, slot (i / 32) % 8. Of each: 256 low - 1 with the least c behind it, 256 (best[i] -
        // best[j - 1]) + 255, and how far back it is. Their product and sum is 256 times what it saves, and 255 less
        // the distance, so that the largest is the best cut with the shortest last run. (It is never below 0 for the
        // last start, and a saving grows by at most one c a step.)
        int low[8], rel[8], far[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            low[k] = 0;
            rel[k] = -1;
            far[k] = 0;
        }
        int next = m > 1 ? 256 * c[0] - 1 : 0;
        for (int j0 = 0; j0 < m; j0 += 256) {
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8)  // the slot of the starts that this stretch of 32 steps adds
                for (int l = 0; l < 32; ++l) {
                    const int i = j0 + 32 * k8 + l;  // the step's new start; j = i + 1
                    if (i >= m) break;
                    const int between = next;  // to the sequence before
                    next = 256 * c[i] - 1;
                    int key = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        low[k] = i > 0 ? min(low[k], between) : 0;
                        ++far[k];
                        if (k == k8 && lane == l) {
                            low[k] = 256 * kMost - 1;
                            rel[k] = 255;
                            far[k] = 0;
                        }
                        key = max(key, rel[k] + far[k] * low[k]);
                    }
                    key = __reduce_max_sync(0xffffffffu, key);
                    if (lane == 0) back[i] = (uint8_t)(255 - (key & 255));
#pragma unroll
                    for (int k = 0; k < 8; ++k) rel[k] -= key & ~255;
                }
        }
        __syncwarp();
        if (lane == 0) {
            int runs = 0;
            for (int j = m; j > 0;) {
                j -= back[j - 1] + 1;
                starts[runs++] = j;
            }
            s_runs = runs;
        }
    }
    __syncthreads();
    for (int r = warp; r < s_runs; r += kThreads / 32) {  // from the last run to the first
        const int lo = starts[r], hi = r ? starts[r - 1] : m;
        int least = kMost;
        for (int i = lo + lane; i < hi - 1; i += 32) least = min(least, c[i]);
        least = __reduce_min_sync(0xffffffffu, least);
        if (hi - lo < 2 || least == 0) continue;
        const int s0 = busy[lo], s1 = busy[hi - 1] + 1;
        for (int s = s0 + lane; s < s1; s += 32) {
            first[s] = s0;
            end[s] = s1;
            shared[s] = least << a.c.page_shift;
        }
    }
}

}  // namespace

size_t cache_prefixes_scratch_bytes(int n_seqs) { return sizeof(int) * (size_t)n_seqs; }
int cache_prefixes_most_seqs() { return 1 << 14; }

cudaError_t launch_cache_prefixes(const CachePrefixArgs& a, cudaStream_t st, int* launches) {
    const int n = a.c.n_seqs, per = kThreads / 32;
    alike_kernel<<<(n + per - 1) / per, kThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const size_t smem = cut_smem(n);
    if (smem > 48 * 1024) {  // (what the longest call needs, whatever this one does: calls of several threads set the same)
        e = cudaFuncSetAttribute(cut_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cut_smem(cache_prefixes_most_seqs()));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, cut_kernel, a);
    if (e == cudaSuccess) *launches += 2;
    return e;
}

}  // namespace bdlm
