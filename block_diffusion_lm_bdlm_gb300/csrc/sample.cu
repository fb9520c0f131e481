// sample.cu - a token for each row of logits, from one random number per row.
//
// Mathematics. With weights w_i = e^((x_i - m) / T), tokens ordered by falling
// logit and among equals by number: top-k keeps the first k; top-p of those
// the ones whose predecessors weigh less than p of what they weigh together;
// min-p those with w >= min_p. All three cut the same order, so what is kept is
// every token above some logit and the first n of those that have it (the cut).
// The token is the first kept one, by number, at which the sum of the kept
// weights passes u times all of it.
//
// Which token that is must not depend on roundings. Sums are first taken from
// the quick weights (sample.cuh), whose error is bounded: where the bound says
// that the decision stands, it does; else it is made from the exact ones. Few
// tokens are near the top of a usual row, so cuts are found from exact weights
// at once.
//
// One cluster of CTAs takes one row. Each CTA copies its part of the row to
// shared memory, where every later pass reads it: the row comes from memory
// once. Passes: the largest logit; sums of the quick weights; for a cut, the
// weights (or for top-k numbers) of the tokens in bins of falling logit, where
// only those bins are filled that the threads' largest logits cannot rule out,
// and the bin with the cut again in finer ones until it is a single logit; the
// kept weights of each warp's part; the tokens of the one part in which the sum
// passes u.
//
// Bound. Memory, for peaked rows; each pass is 64 KB from shared memory and 1
// to 8 instructions a logit. What it takes besides are five to ten barriers of
// the cluster, which the other clusters on the SM fill.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sample.cuh"

namespace bdlm {
namespace {

using namespace sample;
namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;
constexpr int kMaxCtas = 8;
constexpr float kBinsPerOctave = 8.f;  // bins of the first level: an eighth of a factor of two in weight
constexpr float kGreedyBelow = 0x1p-20f;
constexpr float kHottest = 0x1p40f;

template <typename T>
struct Type;
template <>
struct Type<float> {
    static constexpr int VE = 4, SHIFT = 0;
};
template <>
struct Type<__nv_bfloat16> {
    static constexpr int VE = 8, SHIFT = 16;  // low bits of its values as floats that say nothing
};
template <>
struct Type<__half> {
    static constexpr int VE = 8, SHIFT = 13;
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[Type<T>::VE]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            x[i] = __uint_as_float(w[i]);
        } else if constexpr (Type<T>::SHIFT == 16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
// The largest value of a vector; NaN counts as nothing.
template <typename T>
__device__ __forceinline__ float top_of(const uint4& v) {
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else if constexpr (Type<T>::SHIFT == 16) {
        const __nv_bfloat162 *a = reinterpret_cast<const __nv_bfloat162*>(&v);
        const __nv_bfloat162 y = __hmax2(__hmax2(a[0], a[1]), __hmax2(a[2], a[3]));
        return fmaxf(__low2float(y), __high2float(y));
    } else {
        const __half2* a = reinterpret_cast<const __half2*>(&v);
        const __half2 y = __hmax2(__hmax2(a[0], a[1]), __hmax2(a[2], a[3]));
        return fmaxf(__low2float(y), __high2float(y));
    }
}
template <typename T>
__device__ __forceinline__ T value_of(float x) {
    if constexpr (sizeof(T) == 4) return x;
    else if constexpr (Type<T>::SHIFT == 16) return __float2bfloat16_rn(x);
    else return __float2half_rn(x);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename V>
__device__ __forceinline__ V warp_sum(V x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
template <typename V>
__device__ __forceinline__ V warp_scan(V x) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// What is kept: tokens whose key is above `key`, and the first `ties` that have it.
struct Cut {
    uint32_t key;
    long long ties;
    float x;  // the logit of that key
};

enum : int { COUNT = 0, MASS = 1 };

// What a CTA shows the others of its cluster.
struct Shown {
    double quick[kWarps], whole[kWarps];  // per warp: quick weights at T, at T = 1
    unsigned long long sum[kWarps];       // exact kept weights above the cut
    int ties[kWarps];
    float top;
    unsigned int key_lo, key_hi;
    int done;
};

template <typename T>
struct Row {
    static constexpr int VE = Type<T>::VE, SHIFT = Type<T>::SHIFT;
    uint4* data;       // this CTA's part, as 16-byte vectors
    uint32_t* hist;    // [3][kBins]
    Shown* shown;
    const F2* table;
    unsigned long long* scan;  // [kWarps]
    int* found;
    int nv, vw;  // vectors; vectors of each warp, a multiple of 32
    int C;
    float m, c2;  // largest logit; -2 log2(e) / T
    F2 c;
    float mine;  // largest logit of this thread

    __device__ __forceinline__ static uint32_t key_of(float x) { return order_key(__float_as_uint(x)) >> SHIFT; }
    __device__ __forceinline__ static float at_key(uint32_t k) {
        const uint32_t u = k << SHIFT;
        return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~(u | ((1u << SHIFT) - 1u)));
    }
    __device__ __forceinline__ uint64_t exact(float x) const { return exact_weight(x, m, c, table); }
    // a row's distance from the largest logit in octaves of weight, negative
    __device__ __forceinline__ float octaves(float x) const { return fmaf(-0.5f, x, 0.5f * m) * c2; }
    __device__ __forceinline__ int bin_of(float x) const {
        const float t = octaves(x) * -kBinsPerOctave;
        return t < (float)(kBins - 1) ? (int)t : kBins - 1;
    }
    // f(v, x) for the vectors of this thread; skips those without a logit of at least `least`
    template <typename F>
    __device__ __forceinline__ void each(float least, F f) const {
        const int lane = threadIdx.x & 31, v0 = (threadIdx.x >> 5) * vw, v1 = imin(nv, v0 + vw);
        for (int v = v0 + lane; v < v1; v += 32) {
            const uint4 y = data[v];
            if (!(top_of<T>(y) >= least)) continue;
            float x[VE];
            unpack<T>(y, x);
            f(v, x);
        }
    }
    // Adds up the cluster's bins, in which each thread looks after one; returns this bin's sum and the sum of those
    // before it, and their total. `n` bins are in use. All of the cluster's CTAs have filled theirs.
    template <int MODE>
    __device__ __forceinline__ unsigned long long gather(cg::cluster_group& cl, int n, unsigned long long& before,
                                                         unsigned long long& total) {
        const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
        unsigned long long s = 0;
        if (t < n)
            for (int r = 0; r < C; ++r) {
                const uint32_t* h = cl.map_shared_rank(hist, r);
                if (MODE == COUNT) s += h[t];
                else s += (unsigned long long)h[t] + ((unsigned long long)h[kBins + t] << 15) + ((unsigned long long)h[2 * kBins + t] << 30);
            }
        const unsigned long long in = warp_scan(s);
        if (lane == 31) scan[warp] = in;
        __syncthreads();
        before = in - s;
        total = 0;
        for (int w = 0; w < kWarps; ++w) {
            const unsigned long long y = scan[w];
            if (w < warp) before += y;
            total += y;
        }
        __syncthreads();
        return s;
    }
    template <int MODE>
    __device__ __forceinline__ void clear() {
        for (int i = threadIdx.x; i < (MODE == COUNT ? 1 : 3) * kBins; i += kThreads) hist[i] = 0;
        if (threadIdx.x == 0) *found = kBins;
        __syncthreads();
    }
    template <int MODE>
    __device__ __forceinline__ void add(int b, float x) {
        if (MODE == COUNT) {
            atomicAdd(hist + b, 1u);
        } else {  // 15 bits each, so that 2^17 of them fit
            const uint64_t w = exact(x);
            if (const uint32_t p = (uint32_t)w & 0x7fffu) atomicAdd(hist + b, p);
            if (const uint32_t p = (uint32_t)(w >> 15) & 0x7fffu) atomicAdd(hist + kBins + b, p);
            if (const uint32_t p = (uint32_t)(w >> 30)) atomicAdd(hist + 2 * kBins + b, p);
        }
    }

    // The cut of the tokens from key `floor` on at `target` (tokens, or weight in units of 2^-44), which is known to
    // within `off`: a token is kept if those before it are less than the target. False if `off` leaves it open.
    template <int MODE>
    __device__ bool select(cg::cluster_group& cl, double target, double off, uint32_t floor, float floor_x, Cut* cut) {
        unsigned long long before, total, s;
        // The threads' largest logits alone reach the target by bin `last`, so the cut lies no further.
        clear<MODE>();
        if (mine > -INFINITY && key_of(mine) >= floor) add<MODE>(bin_of(mine), mine);
        cl.sync();
        s = gather<MODE>(cl, kBins, before, total);
        if ((double)before < target + off && (double)(before + s) >= target + off) *found = threadIdx.x;
        __syncthreads();
        const int last = imin(*found, kBins - 1);
        // no logit below this one lies in bin `last` (c2 is negative; the margin covers roundings)
        const float edge = last == kBins - 1 ? -INFINITY : m + (last + 1.01f) * 2.f / (kBinsPerOctave * c2) - fabsf(m) * 0x1p-20f;
        const float least = fmaxf(edge, floor_x);
        cl.sync();
        clear<MODE>();
        each(least, [&](int, const float(&x)[VE]) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (!(x[e] >= least) || key_of(x[e]) < floor) continue;
                const int b = bin_of(x[e]);
                if (b <= last) add<MODE>(b, x[e]);
            }
        });
        cl.sync();
        s = gather<MODE>(cl, last + 1, before, total);
        if ((double)before < target && (double)(before + s) >= target) {
            *found = threadIdx.x;
            scan[0] = before;
            if ((double)before >= target - off || (double)(before + s) < target + off) *found = kBins + 1;
        }
        __syncthreads();
        const int bin = *found;
        unsigned long long base = scan[0];
        if (bin >= kBins) return false;
        // the keys of that bin
        unsigned lo = 0xffffffffu, hi = 0;
        each(least, [&](int, const float(&x)[VE]) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (!(x[e] >= least) || bin_of(x[e]) != bin) continue;
                const uint32_t k = key_of(x[e]);
                if (k < floor) continue;
                lo = min(lo, k);
                hi = max(hi, k);
            }
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (threadIdx.x == 0) {
            shown->key_lo = 0xffffffffu;
            shown->key_hi = 0;
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            atomicMin(&shown->key_lo, lo);
            atomicMax(&shown->key_hi, hi);
        }
        cl.sync();
        for (int r = 0; r < C; ++r) {
            const Shown* o = cl.map_shared_rank(shown, r);
            lo = min(lo, o->key_lo);
            hi = max(hi, o->key_hi);
        }
        const float x_lo = at_key(lo);
        while (lo < hi) {
            const int shift = imax(0, 32 - __clz(hi - lo) - 9);
            const int n = (int)((hi - lo) >> shift) + 1;
            clear<MODE>();
            each(x_lo, [&](int, const float(&x)[VE]) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if (!(x[e] >= x_lo)) continue;
                    const uint32_t k = key_of(x[e]);
                    if (k < lo || k > hi) continue;
                    add<MODE>((int)((hi - k) >> shift), x[e]);
                }
            });
            cl.sync();
            s = gather<MODE>(cl, n, before, total);
            before += base;
            if ((double)before < target && (double)(before + s) >= target) {
                *found = threadIdx.x;
                scan[0] = before;
                if ((double)before >= target - off || (double)(before + s) < target + off) *found = kBins + 1;
            }
            __syncthreads();
            const int sub = *found;
            base = scan[0];
            cl.sync();  // the bins are filled anew
            if (sub >= kBins) return false;
            hi -= (uint32_t)sub << shift;
            lo = max(lo, hi - ((1u << shift) - 1u));
        }
        cut->key = hi;
        cut->x = at_key(hi);
        const double w = MODE == COUNT ? 1.0 : (double)exact(cut->x);
        const double rest = target - (double)base;
        cut->ties = (long long)ceil(rest / w);
        return off == 0.0 || (ceil((rest - off) / w) == ceil((rest + off) / w) && rest - off > 0.0);
    }

    // Exact weights of the tokens above the cut and the numbers of those at it, per warp, shown to the cluster.
    __device__ __forceinline__ void show_kept(cg::cluster_group& cl, const Cut& cut) {
        unsigned long long s = 0;
        int n = 0;
        each(cut.x, [&](int, const float(&x)[VE]) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const uint32_t k = key_of(x[e]);
                if (k > cut.key && x[e] > -INFINITY) s += exact(x[e]);
                else if (k == cut.key) ++n;
            }
        });
        s = warp_sum(s);
        n = (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
        if ((threadIdx.x & 31) == 0) {
            shown->sum[threadIdx.x >> 5] = s;
            shown->ties[threadIdx.x >> 5] = n;
        }
        cl.sync();
    }
    // The weight of what the cut keeps.
    __device__ __forceinline__ unsigned long long kept_weight(cg::cluster_group& cl, const Cut& cut) {
        unsigned long long s = 0;
        long long n = 0;
        for (int r = 0; r < C; ++r) {
            const Shown* o = cl.map_shared_rank(shown, r);
            for (int w = 0; w < kWarps; ++w) {
                s += o->sum[w];
                n += o->ties[w];
            }
        }
        n = n < cut.ties ? n : cut.ties;
        return s + (unsigned long long)n * exact(cut.x);
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
    constexpr int VE = Type<T>::VE;
    extern __shared__ uint4 s_data[];
    __shared__ Shown s_shown;
    __shared__ uint32_t s_hist[3 * kBins];
    __shared__ F2 s_table[kTable];
    __shared__ unsigned long long s_scan[kWarps];
    __shared__ float s_top[kWarps];
    __shared__ int s_found;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), row = blockIdx.x / a.ctas;
    if (a.now && __ldg(a.now + row) != a.want) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < kTable) {
        constexpr F2 t[kTable] = {BDLM_POW2_TABLE};
        F2 v = t[0];
#pragma unroll
        for (int i = 1; i < kTable; ++i)
            if (tid == i) v = t[i];
        s_table[tid] = v;
    }
    const int first = rank * a.per, n = imax(0, imin(a.per, a.vocab - first));
    const T* src = static_cast<const T*>(a.x) + (long long)row * a.stride + first;
    const int skew = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));  // elements before ours in the first vector

    Row<T> R;
    R.data = s_data;
    R.hist = s_hist;
    R.shown = &s_shown;
    R.table = s_table;
    R.scan = s_scan;
    R.found = &s_found;
    R.nv = n ? (skew + n + VE - 1) / VE : 0;
    R.vw = ((R.nv + kWarps - 1) / kWarps + 31) & ~31;
    R.C = a.ctas;
    const int v0 = warp * R.vw, v1 = imin(R.nv, v0 + R.vw);
    // Each thread copies the vectors that it will read, so it need only wait for its own.
    for (int v = v0 + lane; v < v1; v += 32) {
        const int e0 = v * VE - skew;
        if (e0 >= 0 && e0 + VE <= n) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(s_data + v)), "l"(src + e0)
                         : "memory");
        } else {  // a vector that is not all ours: what is not weighs nothing
            T* dst = reinterpret_cast<T*>(s_data + v);
#pragma unroll
            for (int e = 0; e < VE; ++e) dst[e] = e0 + e >= 0 && e0 + e < n ? src[e0 + e] : value_of<T>(-INFINITY);
        }
    }
    const float temp = a.temperature ? __ldg(a.temperature + row) : a.temperature_all;
    const int top_k = a.top_k ? __ldg(a.top_k + row) : a.top_k_all;
    const float top_p = a.top_p ? __ldg(a.top_p + row) : a.top_p_all;
    const float min_p = a.min_p ? __ldg(a.min_p + row) : a.min_p_all;
    const float u = fminf(fmaxf(__ldg(a.u + row), 0.f), 1.f);
    const bool greedy = !(temp >= kGreedyBelow);
    const double cd = 2.8853900817779268 / (double)(greedy ? 1.f : fminf(temp, kHottest));
    R.c = F2{(float)cd, (float)(cd - (double)(float)cd)};
    R.c2 = -(float)cd;
    asm volatile("cp.async.wait_all;" ::: "memory");

    // ---- the largest logit
    R.mine = -INFINITY;
    for (int v = v0 + lane; v < v1; v += 32) R.mine = fmaxf(R.mine, top_of<T>(s_data[v]));
    {
        const float x = warp_max(R.mine);
        if (lane == 0) s_top[warp] = x;
        __syncthreads();
        if (tid == 0) {
            float y = s_top[0];
            for (int w = 1; w < kWarps; ++w) y = fmaxf(y, s_top[w]);
            s_shown.top = y;
        }
        cl.sync();
        R.m = -INFINITY;
        for (int r = 0; r < a.ctas; ++r) R.m = fmaxf(R.m, cl.map_shared_rank(&s_shown, r)->top);
    }
    if (R.m == -INFINITY) {  // nothing is left to choose from
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            a.logprob[row] = -INFINITY;
        }
        cl.sync();  // the others may still read what this CTA shows
        return;
    }
    if (R.m == INFINITY) {  // the infinite logits share everything
        R.mine = -INFINITY;
        for (int v = v0 + lane; v < v1; v += 32) {
            T* x = reinterpret_cast<T*>(s_data + v);
            for (int e = 0; e < VE; ++e) {
                const bool top = (float)x[e] == INFINITY;
                x[e] = value_of<T>(top ? 0.f : -INFINITY);
                if (top) R.mine = 0.f;
            }
        }
        R.m = 0.f;
    }

    // ---- sums of the quick weights, at T = 1 for the log-probability and, where they are asked for, at T
    const bool by_k = !greedy && top_k > 0 && top_k < a.vocab, by_p = !greedy && top_p < 1.f, by_min = !greedy && min_p > 0.f;
    const bool quick = !greedy && !by_k && (by_p || !by_min);
    const bool two = quick && temp != 1.f;
    double quick_z = 0.0, whole_z = 0.0;
    for (int turn = 0;; ++turn) {
        const float half_m = 0.5f * R.m, c1 = -2.8853900817779268f;
        float s1 = 0.f, st = 0.f;
        for (int v = v0 + lane; v < v1; v += 32) {
            float x[VE], y = 0.f, yt = 0.f;
            unpack<T>(s_data[v], x);
#pragma unroll
            for (int e = 0; e < VE; e += 2) {
                const float h0 = fmaf(-0.5f, x[e], half_m), h1 = fmaf(-0.5f, x[e + 1], half_m);
                y += ex2(h0 * c1) + ex2(h1 * c1);
                if (two) yt += ex2(h0 * R.c2) + ex2(h1 * R.c2);
            }
            s1 += y;
            st += yt;
        }
        const double w1 = warp_sum((double)s1), wt = two ? warp_sum((double)st) : w1;
        if (lane == 0) {
            s_shown.whole[warp] = w1;
            s_shown.quick[warp] = wt;
        }
        cl.sync();
        whole_z = quick_z = 0.0;
        for (int i = lane; i < a.ctas * kWarps; i += 32) {
            const Shown* o = cl.map_shared_rank(&s_shown, i / kWarps);
            whole_z += o->whole[i % kWarps];
            quick_z += o->quick[i % kWarps];
        }
        whole_z = warp_sum(whole_z);
        quick_z = warp_sum(quick_z);
        if (whole_z == whole_z || turn == 1) break;
        // a NaN counts as a logit of -infinity
        cl.sync();
        for (int v = v0 + lane; v < v1; v += 32) {
            T* x = reinterpret_cast<T*>(s_data + v);
            for (int e = 0; e < VE; ++e)
                if ((float)x[e] != (float)x[e]) x[e] = value_of<T>(-INFINITY);
        }
    }

    // ---- the cut
    Cut cut{0, 0, -INFINITY};
    const double unit = 17592186044416.0;  // 2^44
    if (greedy) {
        cut = Cut{R.key_of(R.m), 1, R.m};
    } else {
        if (by_k) {
            R.template select<COUNT>(cl, (double)top_k, 0.0, 0u, -INFINITY, &cut);
            if (by_p) R.show_kept(cl, cut);
        }
        if (by_p) {
            Cut by{0, 0, -INFINITY};
            double z = quick_z * unit, off = quick_z * unit * kQuick;
            if (by_k) {
                z = (double)R.kept_weight(cl, cut);
                off = 0.0;
            }
            const double p = (double)fmaxf(top_p, 0.f);
            bool sure = false;
            if (p == 0.0) {
                by = Cut{R.key_of(R.m), 1, R.m};
                sure = true;
            } else if (off == 0.0 || p * off < 0.25 * p * z) {
                sure = R.template select<MASS>(cl, p * z, p * off, cut.key, cut.x, &by);
            }
            if (!sure) {  // the sum of all weights again, exactly
                cl.sync();
                R.show_kept(cl, cut);
                z = (double)R.kept_weight(cl, cut);
                R.template select<MASS>(cl, p * z, 0.0, cut.key, cut.x, &by);
            }
            if (by.key > cut.key || !by_k) cut = by;
            else cut.ties = by.ties < cut.ties ? by.ties : cut.ties;
        }
        if (by_min) {
            const double thr = (double)R.m + (double)fminf(temp, kHottest) * log((double)fminf(min_p, 1.f));
            const float x = fminf(__double2float_ru(thr), R.m);
            // the least value of the type that is not below it
            uint32_t k = R.key_of(x);
            if (R.at_key(k) < x) ++k;
            if (k > cut.key) cut = Cut{k, 1LL << 40, R.at_key(k)};
        }
    }

    // ---- the token
    int token = -1;
    float at = 0.f;
    bool mine = false;
    bool done = false;
    if (!greedy && !by_k && !by_p && !by_min) {
        // all tokens, by quick weights
        const double target = (double)u * quick_z, slack = 2.0 * kQuick * quick_z;
        double sum = 0.0;
        int who = -1;
        double base = 0.0;
        for (int i = 0; i < a.ctas * kWarps; ++i) {
            const double y = cl.map_shared_rank(&s_shown, i / kWarps)->quick[i % kWarps];
            if (who < 0 && sum + y > target) {
                who = i;
                base = sum;
            }
            sum += y;
        }
        if (tid == 0) s_shown.done = 0;
        __syncthreads();
        if (who >= 0 && who == rank * kWarps + warp) {
            for (int vb = v0; vb < v1; vb += 32) {
                const int v = vb + lane;
                float x[VE], w[VE];
                double s = 0.0;
                if (v < v1) {
                    unpack<T>(s_data[v], x);
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        w[e] = ex2(fmaf(-0.5f, x[e], 0.5f * R.m) * R.c2);
                        s += w[e];
                    }
                }
                const double in = warp_scan(s) + base;
                const unsigned hit = __ballot_sync(0xffffffffu, in > target);
                if (hit) {
                    if (lane == __ffs(hit) - 1) {
                        double run = in - s;
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            if (token < 0 && run + w[e] > target) {
                                token = first + v * VE + e - skew;
                                at = x[e];
                                mine = run < target - slack && run + w[e] > target + slack;
                            }
                            run += w[e];
                        }
                        s_shown.done = mine;
                    }
                    break;
                }
                base = __shfl_sync(0xffffffffu, in, 31);
            }
        }
        cl.sync();
        for (int r = 0; r < a.ctas; ++r) done = done || cl.map_shared_rank(&s_shown, r)->done;
        if (!done) {
            token = -1;
            mine = false;
        }
    }
    if (!done) {
        cl.sync();
        R.show_kept(cl, cut);
        const unsigned long long tie_w = cut.ties ? R.exact(cut.x) : 0;
        const unsigned long long all = R.kept_weight(cl, cut);
        const double target = (double)u * (double)all;
        // the part in which the sum passes the target; if roundings (or u = 1) leave none, the last that weighs anything
        unsigned long long sum = 0, base = 0;
        long long ties = 0;
        int who = -1, allowed = 0;
        bool passed = false;
        for (int i = 0; i < a.ctas * kWarps; ++i) {
            const Shown* o = cl.map_shared_rank(&s_shown, i / kWarps);
            const int have = o->ties[i % kWarps];
            const long long rest = cut.ties - ties;
            const int take = rest <= 0 ? 0 : rest < have ? (int)rest : have;
            const unsigned long long y = o->sum[i % kWarps] + (unsigned long long)take * tie_w;
            if (!passed && y > 0) {
                who = i;
                base = sum;
                allowed = take;
                passed = (double)(sum + y) > target;
            }
            sum += y;
            ties += have;
        }
        if (who == rank * kWarps + warp) {
            int last_token = -1;
            float last_at = 0.f;
            for (int vb = v0; vb < v1; vb += 32) {
                const int v = vb + lane;
                float x[VE];
                unsigned long long w[VE], s = 0;
                int tied = 0;
                if (v < v1) {
                    unpack<T>(s_data[v], x);
#pragma unroll
                    for (int e = 0; e < VE; ++e) tied += R.key_of(x[e]) == cut.key;
                }
                int before = warp_scan(tied);
                const int all_tied = __shfl_sync(0xffffffffu, before, 31);
                before -= tied;
                if (v < v1) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const uint32_t k = R.key_of(x[e]);
                        w[e] = 0;
                        if (k > cut.key) w[e] = R.exact(x[e]);
                        else if (k == cut.key) w[e] = before++ < allowed ? tie_w : 0;
                        s += w[e];
                    }
                }
                allowed -= all_tied;
                const unsigned long long in = warp_scan(s) + base;
                const unsigned hit = __ballot_sync(0xffffffffu, (double)in > target);
                if (v < v1 && (!hit || lane == __ffs(hit) - 1)) {
                    unsigned long long run = in - s;
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        run += w[e];
                        if (w[e] > 0 && !mine) {
                            last_token = first + v * VE + e - skew;
                            last_at = x[e];
                            mine = hit && (double)run > target;
                        }
                    }
                }
                if (hit) break;
                base = __shfl_sync(0xffffffffu, in, 31);
            }
            if (!__any_sync(0xffffffffu, mine)) {  // the last token that weighs anything
                const int most = (int)__reduce_max_sync(0xffffffffu, (unsigned)(last_token + 1)) - 1;
                mine = last_token == most;
            }
            token = last_token;
            at = last_at;
        }
    }
    if (mine) {
        a.token[row] = token;
        a.logprob[row] = (float)((double)at - (double)R.m - log(whole_z));
    }
    cl.sync();  // no CTA leaves while another may read what it shows
}

template <typename T>
cudaError_t launch(SampleArgs a, int num_sms, cudaStream_t st, int* launches) {
    constexpr int VE = Type<T>::VE;
    // A CTA's part of a row: at most 64 KB, so that three CTAs share an SM; parts of a lone row may be smaller, so that
    // more SMs take part, but a warp should have a vector for each lane.
    auto parts = [&](int c) { return ((a.vocab + c - 1) / c + 63) / 64 * 64; };
    int c = 1;
    while (c < kMaxCtas && (size_t)parts(c) * sizeof(T) > 65536) c *= 2;
    while (c < kMaxCtas && (long long)a.rows * c * 2 <= num_sms && parts(c) > kThreads * VE) c *= 2;
    a.ctas = c;
    a.per = parts(c);
    const size_t smem = ((size_t)a.per / VE + 1) * 16;
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.rows * c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)c;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace

cudaError_t launch_sample(SampleArgs a, int dtype, int num_sms, cudaStream_t st, int* launches) {
    switch (dtype) {
        case 0: return launch<__nv_bfloat16>(a, num_sms, st, launches);
        case 1: return launch<float>(a, num_sms, st, launches);
        default: return launch<__half>(a, num_sms, st, launches);
    }
}

}  // namespace bdlm
