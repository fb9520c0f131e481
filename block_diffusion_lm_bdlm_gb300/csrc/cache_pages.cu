// cache_pages.cu - reserve, fork and compact: which pages are live, which free
// ones are taken, and the copies that follow.
//
// A plan kernel does the bookkeeping of all three calls as one cluster of
// eight CTAs: clear the counts, count how many sequences name each page, rank
// the pages (free ones, or for compact the holes and the pages that move) with
// a prefix sum, check that the call can be done, and only then write table and
// lens. Its phases meet at the cluster's hardware barrier, which also orders
// their global reads and writes, so one launch does what would otherwise take
// one for each phase; it moves a few bytes per page and is bound by latency
// (about 13 us for 256 sequences over 16k positions each).
// A copy kernel then moves the pages of fork and compact, one warp for each
// (copy, layer, K or V, head): a run of contiguous bytes, eight 16-byte loads
// per lane in flight. It is launched with programmatic dependence, so that its
// CTAs are there when the plan ends. Bound by memory: 128 forks of a part of a
// page in 32 layers move 1.2 GB in 165 us (7.2 TB/s, more than a plain copy's
// 6.8, since some of it stays in L2), a compaction of 8 layers 1.05 GB in 182
// us with its plan.
#include <cooperative_groups.h>

#include "cache.cuh"

namespace bdlm {
namespace {

namespace cg = cooperative_groups;

// CTAs of the plan: 8, 4, 2 take 14.6, 16.0, 20.1 us for reserving a block for 256 sequences, 15.0, 13.1, 13.5 for one
// fork into four, 183.5, 181.8, 182.5 for a compaction that moves 0.5 GB (with the calls' copies): more CTAs are worth
// it where there are many pages.
constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
static_assert(kPlanThreads == 32 * 32, "block_scan scans the sums of 32 warps");
constexpr int kAll = kCluster * kPlanThreads;
constexpr int kCopyThreads = 256;

struct Scratch {
    int* n_copies;  // [1]
    int* refused;   // [1] 0, or 1 + the item that the third phase refuses; then padding
    long long* totals;  // [2][kCluster] pages needed, pages free, of each CTA's run
    int* count;     // [n_pages] sequences that name the page
    int* rank;      // [n_pages] free pages in order (reserve, fork); new number of a page that moves (compact)
    int* src;       // [max(n_pages, n_seqs)] copies
    int* dst;
    int* rows;      // rows that a copy takes
    int* child;     // [n_seqs] times a sequence is named as a child
};

__host__ __device__ __forceinline__ Scratch carve(int* p, int n_pages, int n_seqs) {
    Scratch s;
    const long long m = n_pages > n_seqs ? n_pages : n_seqs;
    s.n_copies = p;
    s.refused = p + 1;
    s.totals = reinterpret_cast<long long*>(p + 32);
    s.count = p + 64;
    s.rank = s.count + n_pages;
    s.src = s.rank + n_pages;
    s.dst = s.src + m;
    s.rows = s.dst + m;
    s.child = s.rows + m;
    return s;
}

// Sum of x over the CTA before this thread; *total gets the CTA's sum.
template <typename T>
__device__ T block_scan(T x, T* total, T* buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) buf[warp] = v;
    __syncthreads();
    T w = buf[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    const T before = __shfl_sync(0xffffffffu, w, warp) - __shfl_sync(0xffffffffu, buf[lane], warp);
    *total = __shfl_sync(0xffffffffu, w, 31);
    __syncthreads();
    return before + v - x;
}

__device__ __forceinline__ int pages_of(int len, int shift) { return (int)(((long long)len + (1 << shift) - 1) >> shift); }

// Each CTA of the cluster takes a run of consecutive items; returns the run.
__device__ __forceinline__ void run_of(int n, int rank, int* lo, int* hi) {
    const int per = (n + kCluster - 1) / kCluster;
    *lo = imin(n, rank * per);
    *hi = imin(n, *lo + per);
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads, 1) plan_kernel(const CachePagesArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ int buf[32];
    __shared__ long long wide[32];
    const CacheView& c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, rank = (int)cluster.block_rank();
    const int gtid = rank * kPlanThreads + tid, gwarp = gtid >> 5;
    const int shift = c.page_shift, cap = c.max_pages;
    const int split = imax(1, kAll / 32 / c.n_seqs);  // warps that share the entries of a sequence
    const Scratch s = carve(a.scratch, c.n_pages, c.n_seqs);

    // ---- clear
    for (int i = gtid; i < c.n_pages; i += kAll) s.count[i] = 0;
    for (int i = gtid; i < c.n_seqs; i += kAll) s.child[i] = 0;
    if (gtid == 0) {
        a.hdr->error = DEV_OK;
        a.hdr->info = 0;
        *s.n_copies = 0;
        *s.refused = 0;
    }
    cluster.sync();

    // ---- check the lengths and entries, count the pages' users
    for (int u = gwarp; u < c.n_seqs * split; u += kAll / 32) {
        const int q = u / split, first = (u - q * split) * 32 + lane;
        int len = __ldcg(c.lens + q);
        bool bad = len < 0 || pages_of(len, shift) > cap;
        if (a.op == PAGES_RESERVE) {
            const int want = __ldg(a.new_lens + q);
            bad = bad || want < 0 || pages_of(want, shift) > cap;
            len = imin(len, want);  // pages that are given up are free
        }
        if (!bad) {
            const int n = pages_of(len, shift);
#pragma unroll 4
            for (int i = first; i < n; i += 32 * split) {
                const int id = __ldcg(c.table + (long long)q * c.max_pages + i);
                if (id < 0 || id >= c.n_pages) bad = true;
                else atomicAdd(s.count + id, 1);
            }
        }
        if (bad) set_error(a.hdr, DEV_CHECK, q);
    }
    if (a.op == PAGES_FORK)
        for (int i = gtid; i < a.n; i += kAll) {
            const int p = __ldg(a.parents + i), k = __ldg(a.children + i);
            bool bad = p < 0 || p >= c.n_seqs || k < 0 || k >= c.n_seqs;
            if (!bad) {
                const int n = a.fork_lens ? __ldg(a.fork_lens + i) : __ldcg(c.lens + p);
                bad = n < 0 || n > __ldcg(c.lens + p) || __ldcg(c.lens + k) != 0 || p == k ||
                      atomicAdd(s.child + k, 1) != 0;
            }
            if (bad) set_error(a.hdr, DEV_CHECK, i);
        }
    cluster.sync();

    // ---- how many pages each item needs, and how many are free: totals of this CTA's runs
    int lo, hi, plo, phi, t;
    run_of(a.op == PAGES_FORK ? a.n : c.n_seqs, rank, &lo, &hi);
    run_of(c.n_pages, rank, &plo, &phi);
    // The same for the whole cluster, which the barriers inside `if (ok)` need: nobody writes the word between the barriers
    // on either side of this read. What this phase itself refuses goes to a word of its own.
    bool ok = __ldcg(&a.hdr->error) == DEV_OK;
    auto need_of = [&](int i) {
        if (a.op == PAGES_COMPACT) return 0;
        if (a.op == PAGES_FORK) {
            const int n = a.fork_lens ? __ldg(a.fork_lens + i) : __ldcg(c.lens + __ldg(a.parents + i));
            return (n & (c.page - 1)) ? 1 : 0;
        }
        return imax(0, pages_of(__ldg(a.new_lens + i), shift) - pages_of(__ldcg(c.lens + i), shift));
    };
    if (ok) {
        long long need = 0, free_pages = 0, sum;  // 64 bits: what is asked for may be far more than there is
        for (int i = lo + tid; i < hi; i += kPlanThreads) need += need_of(i);
        block_scan(need, &sum, wide);
        need = sum;
        for (int i = plo + tid; i < phi; i += kPlanThreads) free_pages += __ldcg(s.count + i) == 0;
        block_scan(free_pages, &sum, wide);
        free_pages = sum;
        if (tid == 0) {
            s.totals[rank] = need;
            s.totals[kCluster + rank] = free_pages;
        }
        if (a.op == PAGES_RESERVE)  // nobody grows inside a page that another sequence reads
            for (int i = lo + tid; i < hi; i += kPlanThreads) {
                const int len = __ldcg(c.lens + i);
                if (__ldg(a.new_lens + i) > len && (len & (c.page - 1)) &&
                    __ldcg(s.count + __ldcg(c.table + (long long)i * c.max_pages + (len >> shift))) > 1)
                    atomicCAS(s.refused, 0, i + 1);
            }
        if (a.op == PAGES_FORK)  // nobody is a parent and a child of one call, and no fork's length is one that the call sets
            for (int i = lo + tid; i < hi; i += kPlanThreads) {
                const long long at = (reinterpret_cast<long long>(a.fork_lens + i) - reinterpret_cast<long long>(c.lens)) / 4;
                if (__ldcg(s.child + __ldg(a.parents + i)) || (a.fork_lens && at >= 0 && at < c.n_seqs && __ldcg(s.child + at)))
                    atomicCAS(s.refused, 0, i + 1);
            }
    }
    cluster.sync();

    // ---- ranks: free pages in order; for compact the new number of every page that moves
    long long need64 = 0;
    int need_before = 0, free_before = 0, all_free = 0;
    const int refused = __ldcg(s.refused);  // the same for the whole cluster: nobody writes it any more
    if (ok)
        for (int i = 0; i < kCluster; ++i) {
            const long long x = __ldcg(s.totals + i), y = __ldcg(s.totals + kCluster + i);
            if (i < rank) { need_before += (int)x; free_before += (int)y; }
            need64 += x;
            all_free += (int)y;
        }
    ok = ok && refused == 0;
    const bool fits = need64 <= all_free;
    const int all_need = fits ? (int)need64 : 0;
    const int live = c.n_pages - all_free;
    if (ok && fits) {
        if (a.op != PAGES_COMPACT) {
            int base = free_before;
            for (int i0 = plo; i0 < phi && base < all_need; i0 += kPlanThreads) {
                const int i = i0 + tid;
                const bool f = i < phi && __ldcg(s.count + i) == 0;
                const int at = base + block_scan((int)f, &t, buf);
                if (f && at < all_need) s.rank[at] = i;
                base += t;
            }
        } else {
            // The k-th hole (free page below `live`) takes the k-th mover (live page from `live` on).
            // With F(i) free pages before page i, a hole at i is number F(i), and a mover at i has
            // i - F(i) live pages before it, so live - 1 - (i - F(i)) movers behind it.
            int base = free_before;
            for (int i0 = plo; i0 < phi; i0 += kPlanThreads) {
                const int i = i0 + tid;
                const bool f = i < phi && __ldcg(s.count + i) == 0;
                const int before = base + block_scan((int)f, &t, buf);
                if (i < phi) {
                    if (f && i < live) s.dst[before] = i;
                    if (i == live) *s.n_copies = before;  // as many pages move as there are holes
                    if (!f && i >= live) s.rank[i] = live - 1 - (i - before);
                }
                base += t;
            }
        }
    }
    if (gtid == 0 && refused) {  // the word is not read again
        a.hdr->error = DEV_CHECK;
        a.hdr->info = refused - 1;
    }
    if (gtid == 0 && ok && !fits) {
        a.hdr->error = DEV_NO_PAGES;
        a.hdr->info = (int)(need64 - all_free > 0x7fffffff ? 0x7fffffff : need64 - all_free);
    }
    cluster.sync();
    if (!ok || !fits) return;  // the same for the whole cluster

    // ---- write
    if (a.op == PAGES_RESERVE) {
        int base = need_before;
        for (int i0 = lo; i0 < hi; i0 += kPlanThreads) {
            const int i = i0 + tid;
            const int n = i < hi ? need_of(i) : 0;
            const int at = base + block_scan(n, &t, buf);
            int* row = i < hi ? c.table + (long long)i * c.max_pages + pages_of(__ldcg(c.lens + i), shift) : nullptr;
            constexpr int kFew = 4;
            if (n <= kFew)
                for (int k = 0; k < n; ++k) row[k] = __ldcg(s.rank + at + k);
            for (unsigned todo = __ballot_sync(0xffffffffu, n > kFew); todo; todo &= todo - 1) {  // the warp together
                const int src = __ffs(todo) - 1, m = __shfl_sync(0xffffffffu, n, src);
                const int* from = s.rank + __shfl_sync(0xffffffffu, at, src);
                int* to = reinterpret_cast<int*>(__shfl_sync(0xffffffffu, reinterpret_cast<long long>(row), src));
#pragma unroll 4
                for (int k = lane; k < m; k += 32) to[k] = __ldcg(from + k);
            }
            if (i < hi) c.lens[i] = __ldg(a.new_lens + i);
            base += t;
        }
        return;
    }
    if (a.op == PAGES_FORK) {
        int base = need_before;
        for (int i0 = lo; i0 < hi; i0 += kPlanThreads) {
            const int i = i0 + tid;
            const int n = i < hi ? need_of(i) : 0;
            const int at = base + block_scan(n, &t, buf);
            if (n) {
                const int len = a.fork_lens ? __ldg(a.fork_lens + i) : __ldcg(c.lens + __ldg(a.parents + i));
                const int e = len >> shift, id = __ldcg(s.rank + at);
                s.src[at] = __ldcg(c.table + (long long)__ldg(a.parents + i) * c.max_pages + e);
                s.dst[at] = id;
                s.rows[at] = len & (c.page - 1);
                c.table[(long long)__ldg(a.children + i) * c.max_pages + e] = id;
            }
            base += t;
        }
        const int share = imax(1, kAll / 32 / imax(1, a.n));
        for (int u = gwarp; u < a.n * share; u += kAll / 32) {
            const int i = u / share, part = u - i * share;
            const int p = __ldg(a.parents + i), k = __ldg(a.children + i);
            const int len = a.fork_lens ? __ldg(a.fork_lens + i) : __ldcg(c.lens + p);
            const int* from = c.table + (long long)p * c.max_pages;
            int* to = c.table + (long long)k * c.max_pages;
#pragma unroll 4
            for (int e = part * 32 + lane; e < len >> shift; e += 32 * share) to[e] = __ldcg(from + e);
            if (part == 0 && lane == 0) c.lens[k] = len;
        }
        if (gtid == 0) *s.n_copies = all_need;
        return;
    }
    // compact: the mover with r movers behind it is number moves - 1 - r
    const int moves = __ldcg(s.n_copies);  // 0 without a free page
    for (int i = imax(plo, live) + tid; i < phi; i += kPlanThreads)
        if (__ldcg(s.count + i) != 0) {
            const int k = moves - 1 - __ldcg(s.rank + i), to = __ldcg(s.dst + k);
            s.src[k] = i;
            s.rows[k] = c.page;
            s.rank[i] = to;
        }
    if (gtid == 0 && a.n_live) *a.n_live = live;
    cluster.sync();
    for (int u = gwarp; u < c.n_seqs * split; u += kAll / 32) {
        const int q = u / split, n = pages_of(__ldcg(c.lens + q), shift);
        int* row = c.table + (long long)q * c.max_pages;
#pragma unroll 4
        for (int i = (u - q * split) * 32 + lane; i < n; i += 32 * split) {
            const int id = __ldcg(row + i);
            if (id >= live) row[i] = __ldcg(s.rank + id);
        }
    }
}

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CachePagesArgs a) {
    const CacheView& c = a.c;
    const Scratch s = carve(a.scratch, c.n_pages, c.n_seqs);
    const int lane = threadIdx.x & 31;
    const long long per = 2LL * c.n_layers * c.Hk;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the plan's writes
    const long long total = __ldcg(s.n_copies) * per;
    const long long stride = (long long)gridDim.x * (kCopyThreads / 32);
    for (long long u = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < total; u += stride) {
        const int i = (int)(u / per);
        int rest = (int)(u - i * per);
        const int h = rest % c.Hk;
        rest /= c.Hk;
        const int layer = rest >> 1;
        const int src = __ldcg(s.src + i), dst = __ldcg(s.dst + i), rows = __ldcg(s.rows + i);
        const long long from = ((long long)layer * c.n_pages + src) * c.Hk + h;
        const long long to = ((long long)layer * c.n_pages + dst) * c.Hk + h;
        uint8_t* base = (rest & 1) ? c.v : c.k;
        float* scales = (rest & 1) ? c.v_scale : c.k_scale;
        const uint4* x = reinterpret_cast<const uint4*>(base + from * c.page * c.D);
        uint4* y = reinterpret_cast<uint4*>(base + to * c.page * c.D);
        const int n = rows * c.D / 16;
        for (int j = lane; j < n; j += 32 * 8) {
            uint4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (j + 32 * e < n) v[e] = ld_stream(x + j + 32 * e);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (j + 32 * e < n) __stcs(y + j + 32 * e, v[e]);
        }
        if (lane == 0) scales[to] = scales[from];
    }
}

}  // namespace

size_t cache_pages_scratch_bytes(int n_pages, int n_seqs) {
    const size_t m = n_pages > n_seqs ? n_pages : n_seqs;
    return 4 * (64 + 2 * (size_t)n_pages + 3 * m + (size_t)n_seqs);
}

cudaError_t launch_cache_pages(const CachePagesArgs& a, int num_sms, cudaStream_t st, int* launches) {
    plan_kernel<<<kCluster, kPlanThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    if (a.op == PAGES_RESERVE) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)num_sms * 4);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, copy_kernel, a);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace bdlm
