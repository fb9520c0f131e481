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
// and compares 256 table entries at a time. The second's recurrence is a chain
// of one step per sequence, of which no step can be shorter than a reduction
// over a warp (22 clocks) and what turns its result into the next one's operand
// (20). One warp does nothing else, in rounds of 16 steps, and looks at the starts
// of the last 32 steps; another works out what those add in each step of the next
// round; and eight, one start to a thread, find for each of them the best of all
// starts further back. 64 sequences take 6.8 us in all, 600 take 29, 73 clocks a
// step. (One warp with eight starts per lane took 10.2 and 48, 155 clocks a step.)
#include "cache.cuh"

namespace bdlm {
namespace {

constexpr int kLongest = 256;
constexpr int kThreads = 256;
constexpr int kCutThreads = 64 + kLongest;  // a warp for the steps, one that prepares them, a thread for each start to go back to
constexpr int kSteps = 16;                  // in a round: half a warp
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
// (c has a place before the first, which brings every round's to a 16-byte boundary, and zeros behind the last for two rounds)
__host__ __device__ constexpr int c_places(int n) { return (n + 1 + 3 * kSteps + 3) / 4 * 4; }
size_t cut_smem(int n) { return 4 * (size_t)c_places(n) + (size_t)n * (4 + 4 + 1); }

__global__ void __launch_bounds__(kCutThreads) cut_kernel(const CachePrefixArgs a) {
    extern __shared__ int4 sm[];
    const int n = a.c.n_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* c = reinterpret_cast<int*>(sm) + 1;
    int* busy = c - 1 + c_places(n);
    int* starts = busy + n;
    uint8_t* back = reinterpret_cast<uint8_t*>(starts + n);
    __shared__ int s_warp[kCutThreads / 32], s_runs, s_bad;
    __shared__ int s_start[2][kSteps], s_grown[2];                   // of rounds in turn
    __shared__ __align__(16) int s_best[2][kLongest / 32][kSteps + 4];  // likewise; eight rows' vectors lie in banks of their own
    __shared__ int s_adds[2][kSteps][32];
    constexpr int kNone = -(1 << 30);
    int *first = a.runs, *end = a.runs + n, *shared = a.runs + 2 * (long long)n;
    if (tid == 0) s_bad = 0x7fffffff;
    for (int s = tid; s < n; s += kCutThreads) {
        first[s] = s;
        end[s] = s + 1;
        shared[s] = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    int m = 0;
    for (int s0 = 0; s0 < n; s0 += kCutThreads) {
        const int s = s0 + tid, x = s < n ? __ldcg(a.scratch + s) : kNoRows;
        if (x == kMalformed) atomicMin(&s_bad, s);
        const unsigned has = __ballot_sync(0xffffffffu, x >= 0);
        if (lane == 0) s_warp[warp] = __popc(has);
        __syncthreads();
        int before = m;
        for (int w = 0; w < kCutThreads / 32; ++w) {
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
    // A start s is held as 256 (best[s] - base) + 255, and 256 low - 1 with the least c behind it. The second times the
    // distance to a step, added to the first, is 256 times what the cut saves, and 255 less the distance, so that the largest
    // is the best cut with the shortest last run. (No value passes 32 bits: a saving grows by at most one c a step, and
    // base is best where the round before began: at most 256 steps behind a start, at most 32 before a step's end.)
    if (warp == 1) c[-1] = 0;
    for (int i = m - 1 + tid; i < m + 3 * kSteps - 1; i += kCutThreads)
        if (i >= 0) c[i] = 0;  // (the last sequence's own, and those behind it)
    for (int i = tid; i < kLongest / 32 * kSteps; i += kCutThreads) s_best[0][i / kSteps][i % kSteps] = kNone;
    __syncthreads();
    auto sixteen = [](const int* from, int (&x)[kSteps]) {
#pragma unroll
        for (int k = 0; k < kSteps; k += 4) {
            const int4 y = *reinterpret_cast<const int4*>(from + k);
            x[k] = y.x;
            x[k + 1] = y.y;
            x[k + 2] = y.z;
            x[k + 3] = y.w;
        }
    };
    // What the starts of the last 32 steps, start s in lane s % 32, add to their first part in the steps from i0 on. Those
    // that are not there yet leave their places to older ones, which do no harm.
    int low = 0;
    auto prepare = [&](int i0, int (&to)[kSteps][32]) {
        int behind[kSteps];
        sixteen(c - 1 + i0, behind);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int far = (i0 + k - lane) & 31;
            low = far == 0 ? 256 * kMost - 1 : min(low, 256 * behind[k] - 1);
            to[k][lane] = far <= i0 + k ? far * low : kNone;
        }
    };
    if (warp == kCutThreads / 32 - 1) prepare(0, s_adds[0]);
    __syncthreads();
    int rel = 0, best = 0, grown = 0;  // the first warp's: best: 256 (best[i] - base); grown: by how much base will move behind the round
    int start = -(1 << 20);            // (the starts' threads) none yet
    for (int round = 0; round * kSteps < m; ++round) {
        const int i0 = round * kSteps, now = round & 1;
        if (warp == 0) {
            // (all that is read is read before the steps, and what is written is kept until they are done: a step then is a
            // reduction and five instructions that wait for one another)
            int before[kSteps], adds[kSteps], own = 0;  // own: of the step whose start this lane has
            sixteen(s_best[now][lane & 7], before);
#pragma unroll
            for (int k = 0; k < kSteps; ++k) adds[k] = s_adds[now][k][lane];
            const int mine = lane - kSteps * now;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                if (mine == k) rel = best + 255;
                const int key = __reduce_max_sync(0xffffffffu, max(before[k], rel + adds[k]));
                if (mine == k) own = key;
                best = key & ~255;
            }
            rel -= grown;  // base becomes the best of this round's beginning
            best -= grown;
            grown = best;
            if (mine >= 0 && mine < kSteps) {
                if (i0 + mine < m) back[i0 + mine] = (uint8_t)(255 - (own & 255));
                s_start[now][mine] = rel;
            }
            if (lane == 0) s_grown[now] = grown;
        } else if (warp <= kLongest / 32) {
            // thread s % 256 of these has start s, from the round behind it on
            int behind[kSteps], own = 0;
            sixteen(c - 1 + i0 + kSteps, behind);
            if (round > 0) {
                const int by = s_grown[now ^ 1], half = (round - 1) % (kLongest / kSteps);  // half a warp begins the last round's starts
                rel -= by;
                if (warp - 1 == half >> 1) {
                    int least = c[i0 - kSteps + lane];  // of those from the lane's on
#pragma unroll
                    for (int x = 1; x < 32; x *= 2) {
                        const int more = __shfl_down_sync(0xffffffffu, least, x);
                        if (lane + x < 32) least = min(least, more);
                    }
                    least = __shfl_sync(0xffffffffu, least, lane % kSteps);
                    if (lane / kSteps == (half & 1)) {
                        start = i0 - kSteps + lane % kSteps;
                        rel = s_start[now ^ 1][lane % kSteps] - by;
                        low = 256 * least - 1;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {  // the next round's steps
                const int far = i0 + kSteps + k - start;
                low = min(low, 256 * behind[k] - 1);
                const int key = __reduce_max_sync(0xffffffffu, far < kLongest ? rel + far * low : kNone);
                if (lane == k) own = key;
            }
            if (lane < kSteps) s_best[now ^ 1][warp - 1][lane] = own;
        } else {
            prepare(i0 + kSteps, s_adds[now ^ 1]);
        }
        __syncthreads();
    }
    if (warp == 0) {
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
    // from the last run to the first, eight threads for each
    for (int r = tid / 8; r < s_runs; r += kCutThreads / 8) {
        const int lo = starts[r], hi = r ? starts[r - 1] : m;
        int least = kMost;
        for (int i = lo + tid % 8; i < hi - 1; i += 8) least = min(least, c[i]);
#pragma unroll
        for (int x = 1; x < 8; x *= 2) least = min(least, __shfl_xor_sync(0xffu << (lane & 24), least, x));
        if (hi - lo < 2 || least == 0) continue;
        const int s0 = busy[lo], s1 = busy[hi - 1] + 1;
        for (int s = s0 + tid % 8; s < s1; s += 8) {
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
    cfg.blockDim = dim3(kCutThreads);
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
