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
// tokens are near the top of a usual row, so their weights are exact at once.
//
// One cluster of CTAs takes one row. Each CTA copies its part of the row to
// shared memory, where every later pass reads it: the row comes from memory
// once. The first pass finds the largest logit, and from the largest of 128
// parts of the row a logit from which on as many tokens as top-k asks for, or
// about 130, will lie; the second takes the sums of the quick weights and lists
// those tokens in the first CTA. If the list has all that may be kept, that CTA
// ranks it and draws, and the others are done. Without cuts the token is where
// the quick sums pass u times all. Else the cut is searched in the whole row:
// bf16 logits are counted by value, of which there are so few that one pass
// gives every later sum; others in bins of falling logit, where only those bins
// are filled that the threads' largest logits cannot rule out, and the bin with
// the cut again in finer ones until it is a single logit. The part in which the
// kept weights pass u times all of them then finds the token.
//
// Bound. No one thing. 512 rows of 131072 bf16 logits, a quarter left out, top-p 0.95
// (104 MB, 15 us of memory, 186 us under the profiler): an SM has a CTA for 55 % of
// that time, between clusters of four that need four free places at once, and then
// issues in 61 % of its slots: 48 instructions a logit. A CTA of a listed row takes
// 31 thousand clocks if it is the first and 21 thousand if not, of which the copy is
// 3.8, the maximum and its barrier 4.9, the sums and the list 6.2, their barrier 4.4,
// ranking and drawing 9.2. One of a row that counts its values goes on for 14 to
// count, 6 to weigh the places, 6 to sum up the cluster's, 8 to cut, and 14 to draw.
// 512 whole rows take 84 us greedy, 99 with top-k 50, 133 without cuts, 171 with top-p
// 0.95 where most rows are listed, 305 where all are counted; of fp16 logits where
// none is listed 566, of fp32 ones 1140 (bins, several passes). One row of 32001 takes
// 10 us. Two CTAs of 512 threads share an SM; three of 256 were no faster on the whole.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <utility>

#include "sample.cuh"

namespace bdlm {
namespace {

using namespace sample;
namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;
constexpr int kMaxCtas = 8;
constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: adding it rounds to whole numbers
constexpr int kWholeBits = 0x4b400000;
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

using u64 = unsigned long long;

// floor and ceiling of f * z, exactly; 0 <= f <= 1, z < 2^63.
__device__ __forceinline__ u64 mul_floor(float f, u64 z, bool up = false) {
    if (f >= 1.f) return z;
    const uint32_t b = __float_as_uint(f);
    const int e = imax((int)(b >> 23), 1);                      // f = mant 2^(e - 150)
    const u64 mant = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
    const u64 lo = mant * z, hi = __umul64hi(mant, z);
    const int s = 150 - e;                                      // 24 <= s < 150
    u64 got, rest;
    if (s >= 128) {
        got = 0;
        rest = lo | hi;
    } else if (s >= 64) {
        got = hi >> (s - 64);
        rest = lo | (hi & ((1ull << (s - 64)) - 1));
    } else {
        got = (hi << (64 - s)) | (lo >> s);
        rest = lo & ((1ull << s) - 1);
    }
    return got + (up && rest ? 1 : 0);
}
__device__ __forceinline__ u64 mul_ceil(float f, u64 z) { return mul_floor(f, z, true); }

constexpr int kList = kThreads;  // listed tokens of a row
constexpr int kParts = kMaxCtas * kWarps;  // maxima, and warps of the largest cluster
static_assert(kParts % 32 == 0, "");
constexpr int kPer = kParts / 32;

enum : int { COUNT = 0, MASS = 1 };

// A cut by value: kept are the logits before place `at` and the first `ties` that have its value x, of weight w each;
// `above`: what those before it weigh.
struct Cut {
    int at;
    long long ties;
    u64 w, above;
    float x;
};
// What the cluster's CTAs tell each other: every CTA has all of it. Entry r * kWarps + w is of warp w of CTA r.
struct All {
    alignas(16) float top[kParts];   // largest logits of the threads in equal groups, 128 in the cluster
    u64 quick[kParts];   // quick weights at T; later exact weights above the cut
    u64 whole[kParts];   // quick weights at T = 1; later exact weights below the cut
    int ties[kParts];    // tokens at the cut
    u64 sums[kMaxCtas][3];  // of each CTA: quick weights at T = 1, at T, and of what it has listed (~0: a NaN)
    int n[kMaxCtas];         // tokens that each CTA has listed
    uint32_t key_lo[kMaxCtas], key_hi[kMaxCtas];
    int done[kMaxCtas];
    int odd[kMaxCtas];  // whether it has a logit without a place
};
// The list of the row's first tokens, in the cluster's first CTA.
struct List {
    uint2 raw[kList];  // key, number; each CTA has an equal part of it
    ulonglong2 tokens[kList], kept[kList];  // order, weight
};
// Bins of a select; the list is done with by then.
struct Bins {
    uint32_t n[kBins];
};
constexpr int kBase = 105 << 7;  // bits of 2^-22 as bf16
// Numbers of the bf16 logits of each value from the largest down, two to a word: 2^10 > |x| > 2^-22, and 0.
constexpr int kValues = 8192;
struct Values {
    uint32_t n[kValues / 2];
};
constexpr int kStretch = kValues / kThreads;  // places that a thread looks after
// What the values before each stretch of places number and weigh, in this CTA and (sum) in the cluster.
struct Upto {
    u64 weight[kThreads + 1], sum_weight[kThreads + 1];
    int count[kThreads + 1], sum_count[kThreads + 1];
};
union Work {
    List list;
    Bins bins;
    Values values;
};

template <typename T>
struct Row {
    static constexpr int VE = Type<T>::VE, SHIFT = Type<T>::SHIFT;
    uint4* data;  // this CTA's part, as 16-byte vectors
    All* all;
    Work* work;
    const F2* table;
    u64* scan;   // [kWarps]
    u64* found;  // [2]
    u64* part;   // [kWarps]
    Upto* upto;
    int nv, vw;  // vectors; vectors of each warp, a multiple of 32
    int C, rank;
    float m, c2;  // largest logit; -2 log2(e) / T
    F2 c;
    float mine;  // largest logit of this thread

    __device__ __forceinline__ static uint32_t key_of(float x) { return order_key(__float_as_uint(x)) >> SHIFT; }
    __device__ __forceinline__ static float at_key(uint32_t k) {
        const uint32_t u = k << SHIFT;
        return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~(u | ((1u << SHIFT) - 1u)));
    }
    __device__ __forceinline__ u64 exact(float x) const { return exact_weight(x, m, c, table); }
    // Distance from the largest logit in bins, and the bin, to which it is rounded (as bits of that plus 1.5 * 2^23).
    __device__ __forceinline__ float bins_off(float x) const {
        return fminf(fmaf(-0.5f, x, 0.5f * m) * (c2 * -kBinsPerOctave), (float)(kBins - 1));
    }
    __device__ __forceinline__ int bin_of(float x) const { return __float_as_int(bins_off(x) + kWhole) - kWholeBits; }
    // No logit of bin b lies above (below) this one. c2 is negative; the margins cover roundings.
    __device__ __forceinline__ float above_bin(int b) const {
        return fminf(m, m + (b - 0.51f) * 2.f / (kBinsPerOctave * c2) + fabsf(m) * 0x1p-20f);
    }
    __device__ __forceinline__ float below_bin(int b) const {
        return b == kBins - 1 ? -INFINITY : m + (b + 0.51f) * 2.f / (kBinsPerOctave * c2) - fabsf(m) * 0x1p-20f;
    }
    // Tells every CTA of the cluster a value for this warp; all lanes hold it.
    template <typename V>
    __device__ __forceinline__ void tell(cg::cluster_group& cl, V* where, V x) const {
        const int lane = threadIdx.x & 31;
        if (lane < C) cl.map_shared_rank(where, lane)[rank * kWarps + (threadIdx.x >> 5)] = x;
    }
    // f(v, x) for the vectors of this thread, without those that have no logit of at least `least`
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
    __device__ __forceinline__ void clear() {
        for (int i = threadIdx.x; i < kBins; i += kThreads) work->bins.n[i] = 0;
        __syncthreads();
    }
    // Counts x in place `at`. MASS: its quick weight in units of 2^-16 of 2^(-bin / 8), at most 2^16.1 of them.
    template <int MODE>
    __device__ __forceinline__ void add(int at, float off_bin) {
        atomicAdd(&work->bins.n[at], MODE == COUNT ? 1u : (uint32_t)(__float_as_int(fmaf(ex2(off_bin * (-1.f / kBinsPerOctave)), 65536.f, kWhole)) - kWholeBits));
    }
    // Adds up the cluster's bins, each thread one, and finds the one in which the sum from `base` on passes the target:
    // its number, and in *before the sum of those before it. Bin i holds weights of octave bin `bin0` + i (MASS, first
    // level) or of `bin0` alone. A target that none passes is taken to be passed by the last bin with anything in it.
    template <int MODE>
    __device__ __forceinline__ int cross(cg::cluster_group& cl, int n, int bin0, bool spread, u64 target, u64 base, u64* before) {
        const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
        u64 s = 0;
        if (t < n) {
#pragma unroll
            for (int r = 0; r < kMaxCtas; ++r)
                if (r < C) s += cl.map_shared_rank(&work->bins, r)->n[t];
        }
        if (MODE == MASS) {
            const int b = spread ? bin0 + t : bin0;
            // 2^16 weights of the bin's largest, 2^(-b / 8), in units of 2^-44
            const int j = -(b & 7) * 2, shift = b >> 3;
            const float top = table[j < -8 ? j + 24 : j + 8].hi;  // 2^(j / 16), or twice that below -8
            const u64 f = (u64)__float2uint_rn(top * 65536.f) << (j < -8 ? 11 : 12);
            s = shift < 44 ? (s * f) >> shift : 0;
        }
        const u64 in = warp_scan(s);
        if (lane == 31) scan[warp] = in;
        if (t == 0) found[0] = 0;
        __syncthreads();
        u64 at = base + in - s;
        for (int w = 0; w < kWarps; ++w)
            if (w < warp) at += scan[w];
        // the bin that passes the target, else the last one with anything in it: the largest of (passes, ~number | number)
        const bool passes = at < target && at + s >= target;
        unsigned key = passes ? 0x80000000u | t : s > 0 ? (unsigned)t + 1 : 0u;
        const unsigned top = __reduce_max_sync(0xffffffffu, key);
        if (lane == 0 && top) atomicMax(reinterpret_cast<unsigned*>(found), top);
        __syncthreads();
        const unsigned got = *reinterpret_cast<unsigned*>(found);
        const int bin = got & 0x80000000u ? (int)(got & 0x7fffffffu) : imax(0, (int)got - 1);
        if (t == bin) found[1] = at;
        __syncthreads();
        *before = found[1];
        return bin;
    }
    // Whether the last cross found a bin that passes.
    __device__ __forceinline__ bool passed() const { return *reinterpret_cast<const unsigned*>(found) & 0x80000000u; }

    // The key of the token at which the sum over falling logits, of tokens (COUNT) or of quick weights (MASS), passes the
    // target; only tokens from logit `floor_x` on count. *before (COUNT): tokens above that key.
    template <int MODE>
    __device__ __forceinline__ uint32_t select(cg::cluster_group& cl, u64 target, float floor_x, u64* before) {
        u64 base;
        int last = kBins - 1;
        cl.sync();
        if (MODE == COUNT && target <= (u64)C * kThreads / 2) {
            // the threads' largest logits alone pass the target by bin `last`, so the cut lies no further
            clear();
            if (mine > -INFINITY) add<MODE>(bin_of(mine), 0.f);
            cl.sync();
            last = cross<MODE>(cl, kBins, 0, true, target, 0, &base);
            if (!passed()) last = kBins - 1;
            cl.sync();
        }
        float least = fmaxf(below_bin(last), floor_x);
        clear();
        each(least, [&](int, const float(&x)[VE]) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (!(x[e] >= least)) continue;
                const float t = bins_off(x[e]), b = t + kWhole;
                add<MODE>(__float_as_int(b) - kWholeBits, t - (b - kWhole));  // (a bin beyond `last` does no harm)
            }
        });
        cl.sync();
        const int bin = cross<MODE>(cl, last + 1, 0, true, target, 0, &base);
        cl.sync();
        // the keys of that bin, coarsely and finer until it is a single one
        least = fmaxf(below_bin(bin), floor_x);
        const float most = above_bin(bin);
        uint32_t lo = key_of(least), hi = key_of(most);
        while (lo < hi) {
            const int shift = imax(0, 32 - __clz(hi - lo) - 9);
            const int n = (int)((hi - lo) >> shift) + 1;
            clear();
            each(least, [&](int, const float(&x)[VE]) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if (!(x[e] >= least && x[e] <= most)) continue;
                    const float t = bins_off(x[e]), b = t + kWhole;
                    const uint32_t k = key_of(x[e]);
                    if (__float_as_int(b) - kWholeBits == bin && k >= lo && k <= hi) add<MODE>((int)((hi - k) >> shift), t - (b - kWhole));
                }
            });
            cl.sync();
            const int sub = cross<MODE>(cl, n, bin, false, target, base, &base);
            hi -= (uint32_t)sub << shift;
            lo = max(lo, hi - ((1u << shift) - 1u));
            cl.sync();  // the bins are filled anew
        }
        *before = base;
        return hi;
    }
    // The least and the largest of the cluster's keys.
    __device__ __forceinline__ void span(cg::cluster_group& cl, uint32_t& lo, uint32_t& hi) {
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        uint32_t* mm = reinterpret_cast<uint32_t*>(found);
        if (threadIdx.x == 0) {
            mm[0] = 0xffffffffu;
            mm[1] = 0;
        }
        __syncthreads();
        const int lane = threadIdx.x & 31;
        if (lane == 0) {
            atomicMin(mm, lo);
            atomicMax(mm + 1, hi);
        }
        __syncthreads();
        if (threadIdx.x < C) {
            All* o = cl.map_shared_rank(all, threadIdx.x);
            o->key_lo[rank] = mm[0];
            o->key_hi[rank] = mm[1];
        }
        cl.sync();
        lo = __reduce_min_sync(0xffffffffu, all->key_lo[lane % C]);
        hi = __reduce_max_sync(0xffffffffu, all->key_hi[lane % C]);
    }

    // The least key above `cut`, or the largest below it, in the row.
    __device__ __forceinline__ uint32_t next_key(cg::cluster_group& cl, uint32_t cut, bool up) {
        uint32_t lo = 0xffffffffu, hi = 0;
        each(-INFINITY, [&](int, const float(&x)[VE]) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const uint32_t k = key_of(x[e]);
                if (k > cut) lo = min(lo, k);
                if (k < cut) hi = max(hi, k);
            }
        });
        span(cl, lo, hi);
        return up ? lo : hi;
    }
    // The least key whose weight is at least w (1 <= w <= 2^44): 32 keys at a time.
    __device__ __forceinline__ uint32_t key_from(u64 w) const {
        const int lane = threadIdx.x & 31;
        uint32_t lo = key_of(-INFINITY), hi = key_of(m);  // of lo the weight is less, of hi it is not
        while (hi - lo > 1) {
            const uint32_t step = (hi - lo - 1) / 32 + 1, k = lo + (uint32_t)(lane + 1) * step;
            const bool has = k >= hi || k < lo || exact(at_key(k)) >= w;
            const int l = __ffs(__ballot_sync(0xffffffffu, has)) - 1;  // (the last lane's key is not below hi)
            const uint32_t top = lo + (uint32_t)(l + 1) * step;
            lo += (uint32_t)l * step;
            hi = top < hi && top > lo ? top : hi;
        }
        return hi;
    }

    // Exact weights of the tokens above key `cut` (in all->quick) and, if they are wanted, below it (all->whole), and the
    // numbers of those at it, of every warp of the cluster.
    __device__ __forceinline__ void weigh(cg::cluster_group& cl, uint32_t cut, bool below) {
        u64 s = 0, z = 0;
        int n = 0;
        const float at = cut ? at_key(cut) : -INFINITY;
        cl.sync();  // what is told is read no more
        each(below ? -INFINITY : at, [&](int, const float(&x)[VE]) {
#pragma unroll
            for (int e = 0; e < VE; e += 2) {
                n += (x[e] == at) + (x[e + 1] == at);
                if (!below && !(x[e] > at || x[e + 1] > at)) continue;
                u64 w0, w1;
                exact_weights(x[e], x[e + 1], m, c, table, w0, w1);
                s += (x[e] > at ? w0 : 0) + (x[e + 1] > at ? w1 : 0);
                if (below) z += (x[e] < at ? w0 : 0) + (x[e + 1] < at ? w1 : 0);
            }
        });
        tell(cl, all->quick, warp_sum(s));
        tell(cl, all->ties, (int)__reduce_add_sync(0xffffffffu, (unsigned)n));
        if (below) tell(cl, all->whole, warp_sum(z));
        cl.sync();
    }
    // Place of a bf16 logit among the values; -1: none.
    __device__ __forceinline__ static int place_of(uint32_t u) {
        const int a = (int)(u & 0x7fffu), r = a - kBase, sign = (int)(u << 16) >> 31;
        return (unsigned)(r - 1) < (unsigned)(kValues / 2 - 1) ? kValues / 2 - 1 - (r ^ sign) : a == 0 ? kValues / 2 - 1 : -1;
    }
    __device__ __forceinline__ static float value_at(int p) {
        const uint32_t u = p < kValues / 2 - 1 ? kValues / 2 - 1 - p + kBase : p == kValues / 2 - 1 ? 0u : 0x8000u + p - kValues / 2 + kBase;
        return __uint_as_float(u << 16);
    }
    // The first place whose value is not above x.
    __device__ __forceinline__ static int place_from(float x) {
        const int r = (int)(__float_as_uint(fabsf(x)) >> 16) - kBase;
        if (x > 0.f) return kValues / 2 - 1 - imax(0, imin(r, kValues / 2 - 1));
        return x == 0.f ? kValues / 2 - 1 : kValues / 2 + imax(0, imin(r, kValues / 2));
    }
    // Counts the values of this CTA's part, and sums up what those before each stretch number and weigh; false if the
    // cluster has a logit without a place. All of the cluster has summed up then.
    __device__ __forceinline__ bool count_values(cg::cluster_group& cl) {
        uint32_t* count = work->values.n;
        for (int i = threadIdx.x; i < kValues / 2; i += kThreads) count[i] = 0;
        __syncthreads();
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, v0 = warp * vw, v1 = imin(nv, v0 + vw);
        bool odd = false;
        for (int v = v0 + lane; v < v1; v += 32) {
            const uint4 y = data[v];
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
                const int p = place_of(u);
                if (p >= 0) atomicAdd(count + (p >> 1), p & 1 ? 0x10000u : 1u);
                else odd = odd || u != 0xff80u;
            }
        }
        const int any = __syncthreads_or(odd);
        if (tid < C) cl.map_shared_rank(all, tid)->odd[rank] = any;
        // of each stretch, kStretch / 2 pairs of places, as many lanes have one pair each
#pragma unroll 1
        for (int q = tid; q < kValues / 2; q += kThreads) {
            const uint32_t y = count[q];
            u64 w0 = 0, w1 = 0, w = 0;
            int n = 0;
            if (__any_sync(0xffffffffu, y)) {
                exact_weights(value_at(2 * q), value_at(2 * q + 1), m, c, table, w0, w1);
                n = (int)((y & 0xffffu) + (y >> 16));
                w = (y & 0xffffu) * w0 + (y >> 16) * w1;
#pragma unroll
                for (int o = 1; o < kStretch / 2; o *= 2) {
                    n += __shfl_xor_sync(0xffffffffu, n, o);
                    w += __shfl_xor_sync(0xffffffffu, w, o);
                }
            }
            if (lane % (kStretch / 2) == 0) {
                upto->sum_weight[q / (kStretch / 2)] = w;
                upto->sum_count[q / (kStretch / 2)] = n;
            }
        }
        __syncthreads();
        const u64 w = upto->sum_weight[tid];
        const int n = upto->sum_count[tid];
        u64 w_in = warp_scan(w);
        int n_in = warp_scan(n);
        if (lane == 31) {
            scan[warp] = w_in;
            part[warp] = (u64)n_in;
        }
        __syncthreads();
        for (int i = 0; i < warp; ++i) {
            w_in += scan[i];
            n_in += (int)part[i];
        }
        upto->weight[tid + 1] = w_in;
        upto->count[tid + 1] = n_in;
        if (tid == 0) {
            upto->weight[0] = 0;
            upto->count[0] = 0;
        }
        cl.sync();
        if (__any_sync(0xffffffffu, all->odd[lane % C])) return false;
        u64 sw = 0;
        int sn = 0;
#pragma unroll
        for (int r = 0; r < kMaxCtas; ++r)
            if (r < C) {
                const Upto* o = cl.map_shared_rank(upto, r);
                sw += o->weight[tid + 1];
                sn += o->count[tid + 1];
            }
        upto->sum_weight[tid + 1] = sw;
        upto->sum_count[tid + 1] = sn;
        if (tid == 0) {
            upto->sum_weight[0] = 0;
            upto->sum_count[0] = 0;
        }
        __syncthreads();
        return true;
    }
    // The place at which the count (MODE COUNT) or the weight passes the target, by every warp for itself.
    template <int MODE>
    __device__ __forceinline__ Cut cut_values(cg::cluster_group& cl, u64 target) {
        const int tid = threadIdx.x, lane = tid & 31;
        const u64 lo = MODE == COUNT ? (u64)upto->sum_count[tid] : upto->sum_weight[tid];
        const u64 hi = MODE == COUNT ? (u64)upto->sum_count[tid + 1] : upto->sum_weight[tid + 1];
        __syncthreads();
        if (lo < target && hi >= target) found[0] = tid;
        __syncthreads();
        // the places of that stretch, one per lane (two lanes' worth of sums: all are kept by every warp)
        const int t = (int)found[0], place = t * kStretch + lane;
        int n = 0;
        u64 w = 0;
        if (lane < kStretch) {
#pragma unroll
            for (int r = 0; r < kMaxCtas; ++r)
                if (r < C) {
                    const uint32_t y = cl.map_shared_rank(&work->values, r)->n[place >> 1];
                    n += (int)(place & 1 ? y >> 16 : y & 0xffffu);
                }
            if (n) w = exact(value_at(place));
        }
        const u64 add = MODE == COUNT ? (u64)n : (u64)n * w, base = MODE == COUNT ? (u64)upto->sum_count[t] : upto->sum_weight[t];
        const u64 in = warp_scan(add) + base, above = warp_scan((u64)n * w) - (u64)n * w + upto->sum_weight[t];
        const int l = __ffs(__ballot_sync(0xffffffffu, in >= target)) - 1;
        Cut cut;
        cut.at = t * kStretch + l;
        cut.x = value_at(cut.at);
        cut.w = __shfl_sync(0xffffffffu, w, l);
        cut.above = __shfl_sync(0xffffffffu, above, l);
        const u64 rest = target - __shfl_sync(0xffffffffu, in - add, l);
        cut.ties = (long long)(MODE == COUNT ? rest : (rest + cut.w - 1) / cut.w);
        return cut;
    }
    // What a cut keeps of CTA `lane`'s tokens: what those before it weigh, and the number of those at it.
    __device__ __forceinline__ u64 kept_of(cg::cluster_group& cl, const Cut& cut, int* tied) const {
        const int lane = threadIdx.x & 31, t = imin(cut.at, kValues) / kStretch, place = t * kStretch + lane;
        u64 s = lane < C ? cl.map_shared_rank(upto, lane)->weight[t] : 0, w = 0;
        if (lane < kStretch && place < imin(cut.at, kValues)) w = exact(value_at(place));
#pragma unroll
        for (int r = 0; r < kMaxCtas; ++r)
            if (r < C) {
                const uint32_t y = w ? cl.map_shared_rank(&work->values, r)->n[place >> 1] : 0;
                const u64 more = warp_sum((u64)(place & 1 ? y >> 16 : y & 0xffffu) * w);
                if (lane == r) s += more;
            }
        *tied = 0;
        if (cut.at < kValues && value_at(cut.at) == cut.x && lane < C) {
            const uint32_t y = cl.map_shared_rank(&work->values, lane)->n[cut.at >> 1];
            *tied = (int)(cut.at & 1 ? y >> 16 : y & 0xffffu);
        }
        return s;
    }
    __device__ __forceinline__ u64 total(const u64* of) const {
        u64 s = 0;
        for (int i = threadIdx.x & 31; i < C * kWarps; i += 32) s += of[i];
        return warp_sum(s);
    }
    __device__ __forceinline__ long long total_ties() const {
        int n = 0;
        for (int i = threadIdx.x & 31; i < C * kWarps; i += 32) n += all->ties[i];
        return (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
    }
    // This warp's kept weight above x, exact or quick, and its numbers of logits that are x.
    template <bool EXACT>
    __device__ __forceinline__ void kept_here(float cut, u64* sum, int* ties) const {
        u64 s = 0;
        float q = 0.f;
        int n = 0;
        each(cut, [&](int, const float(&x)[VE]) {
#pragma unroll
            for (int e = 0; e < VE; e += 2) {
                n += (x[e] == cut) + (x[e + 1] == cut);
                if (!(x[e] > cut || x[e + 1] > cut)) continue;
                if (EXACT) {
                    u64 w0, w1;
                    exact_weights(x[e], x[e + 1], m, c, table, w0, w1);
                    s += (x[e] > cut ? w0 : 0) + (x[e + 1] > cut ? w1 : 0);
                } else {
                    q += (x[e] > cut ? quick(x[e]) : 0.f) + (x[e + 1] > cut ? quick(x[e + 1]) : 0.f);
                }
            }
        });
        *sum = warp_sum(EXACT ? s : (u64)__float2ull_rn(q * 0x1p44f));
        *ties = (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
    }
    __device__ __forceinline__ float quick(float x) const { return ex2(fmaf(-0.5f, x, 0.5f * m) * c2); }
    // The token of this warp's part at which the kept weights, from `base` on, pass the target; `allowed` of those that are
    // cut.x count. The lane that has it returns true; `slack`: it is sure of it by that much.
    template <bool EXACT>
    __device__ __forceinline__ bool walk(float cut, int allowed, u64 tie_w, u64 base, u64 target, u64 slack, int* index, float* at) const {
        const int lane = threadIdx.x & 31, v0 = (threadIdx.x >> 5) * vw, v1 = imin(nv, v0 + vw);
        for (int vb = v0; vb < v1; vb += 32) {
            const int v = vb + lane;
            float x[VE];
            int tied = 0;
#pragma unroll
            for (int e = 0; e < VE; ++e) x[e] = -INFINITY;
            if (v < v1) unpack<T>(data[v], x);
#pragma unroll
            for (int e = 0; e < VE; ++e) tied += x[e] == cut;
            int mine_ = 0;  // of the tied ones, those that count
            if (__any_sync(0xffffffffu, tied)) {
                const int upto = warp_scan(tied);
                mine_ = imax(0, imin(tied, allowed - (upto - tied)));
                allowed -= __shfl_sync(0xffffffffu, upto, 31);
            }
            u64 s = (u64)mine_ * tie_w;
            float q = 0.f;
            if (EXACT) {
#pragma unroll
                for (int e = 0; e < VE; e += 2) {
                    u64 w0, w1;
                    if (!(x[e] > cut || x[e + 1] > cut)) continue;
                    exact_weights(x[e], x[e + 1], m, c, table, w0, w1);
                    s += (x[e] > cut ? w0 : 0) + (x[e + 1] > cut ? w1 : 0);
                }
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) q += x[e] > cut ? quick(x[e]) : 0.f;
                s += __float2ull_rn(q * 0x1p44f);
            }
            const u64 in = warp_scan(s) + base;
            const unsigned hit = __ballot_sync(0xffffffffu, in > target);
            if (hit) {
                bool got = false;
                if (lane == __ffs(hit) - 1) {
                    u64 run = in - s;
#pragma unroll 1
                    for (int e = 0; e < VE; ++e) {
                        const float y = (float)reinterpret_cast<const T*>(data + v)[e];
                        u64 w = 0;
                        if (y > cut) w = EXACT ? exact(y) : (u64)__float2ull_rn(quick(y) * 0x1p44f);
                        else if (y == cut) w = mine_-- > 0 ? tie_w : 0;
                        if (run + w > target) {
                            *index = v * VE + e;
                            *at = y;
                            got = run + slack <= target && run + w > target + slack;
                            break;
                        }
                        run += w;
                    }
                }
                return got;
            }
            base = __shfl_sync(0xffffffffu, in, 31);
        }
        return false;
    }
    __device__ __forceinline__ u64 cta_sum(u64 x) {
        x = warp_sum(x);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) scan[threadIdx.x >> 5] = x;
        __syncthreads();
        u64 s = 0;
        for (int w = 0; w < kWarps; ++w) s += scan[w];
        return s;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
    constexpr int VE = Type<T>::VE;
    extern __shared__ uint4 s_data[];
    __shared__ All s_all;
    __shared__ Work s_work;
    __shared__ F2 s_table[kTable];
    __shared__ u64 s_scan[kWarps], s_found[2];
    __shared__ int s_n, s_nan;
    __shared__ u64 s_part[3][kWarps];
    __shared__ Upto s_upto;
    cg::cluster_group cl = cg::this_cluster();
    // (rows that are left leave with all of their CTAs)
    const int rank = (int)cl.block_rank(), row = blockIdx.x / a.ctas;
    if (a.now && __ldg(a.now + row) != a.want) return;
    auto started = cl.barrier_arrive();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = rank * a.per, n = imax(0, imin(a.per, a.vocab - first));
    const T* src = static_cast<const T*>(a.x) + (long long)row * a.stride + first;
    const int skew = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));  // elements before ours in the first vector

    Row<T> R;
    R.data = s_data;
    R.all = &s_all;
    R.work = &s_work;
    R.table = s_table;
    R.scan = s_scan;
    R.found = s_found;
    R.part = s_part[0];
    R.upto = &s_upto;
    R.nv = n ? (skew + n + VE - 1) / VE : 0;
    R.vw = ((R.nv + kWarps - 1) / kWarps + 31) & ~31;
    R.C = a.ctas;
    R.rank = rank;
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
    // The part that a CTA behind those that run now will read goes to L2.
    if (tid == 0) {
        const long long later = blockIdx.x + a.ahead;
        if (later < (long long)a.rows * a.ctas) {
            const int r = (int)(later / a.ctas);
            const uintptr_t from = reinterpret_cast<uintptr_t>(static_cast<const T*>(a.x) + (long long)r * a.stride + first), at = (from + 15) & ~(uintptr_t)15;
            const uint32_t bytes = (uint32_t)((from + n * sizeof(T) > at ? from + n * sizeof(T) - at : 0) & ~(uintptr_t)15);
            if (bytes && (!a.now || __ldg(a.now + r) == a.want))
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
        }
    }
    if (tid < kTable) {
        constexpr F2 t[kTable] = {BDLM_POW2_TABLE};
        F2 v = t[0];
#pragma unroll
        for (int i = 1; i < kTable; ++i)
            if (tid == i) v = t[i];
        s_table[tid] = v;
    }
    if (tid == 0) {
        s_n = s_nan = 0;
    }
    const float temp = a.temperature ? __ldg(a.temperature + row) : a.temperature_all;
    const int top_k = a.top_k ? __ldg(a.top_k + row) : a.top_k_all;
    const float top_p = a.top_p ? __ldg(a.top_p + row) : a.top_p_all;
    const float min_p = a.min_p ? __ldg(a.min_p + row) : a.min_p_all;
    const float u = fminf(fmaxf(__ldg(a.u + row), 0.f), 1.f);
    const bool greedy = !(temp >= kGreedyBelow) || top_p <= 0.f;  // the first of the largest
    const bool by_k = !greedy && top_k > 0 && top_k < a.vocab, by_p = !greedy && top_p < 1.f, by_min = !greedy && min_p > 0.f;
    const bool cuts = greedy || by_k || by_p || by_min;
    const float T_ = greedy ? 1.f : fminf(temp, kHottest), p = top_p;
    {  // 2 log2(e) / T in two floats: the remainder of the quotient of the high parts, and the low parts
        constexpr float hi = 0x1.715476p+1f, lo = 0x1.4ae0c0p-25f;  // 2 log2(e)
        const float q = __fdiv_rn(hi, T_);
        R.c = F2{q, __fdiv_rn(__fmaf_rn(-q, T_, hi) + lo, T_)};
        R.c2 = -q;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (a.barred >= first && a.barred < first + n) {  // who copied it takes it out
        const int e = a.barred - first + skew, v = e / VE;
        if (v >= v0 && v < v1 && (v & 31) == lane) reinterpret_cast<T*>(s_data)[e] = value_of<T>(-INFINITY);
    }

    // ---- the largest logit
    R.mine = -INFINITY;
    for (int v = v0 + lane; v < v1; v += 32) R.mine = fmaxf(R.mine, top_of<T>(s_data[v]));
    {
        const int groups = kMaxCtas / a.ctas;  // of a warp's lanes
        float x = R.mine;
        for (int o = 1; o < 32 / groups; o *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        cl.barrier_wait(std::move(started));  // every CTA's shared memory is there
        if (lane % (32 / groups) == 0)
            for (int r = 0; r < a.ctas; ++r) cl.map_shared_rank(s_all.top, r)[(rank * kWarps + warp) * groups + lane / (32 / groups)] = x;
    }
    cl.sync();
    float tops[kPer];
    R.m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        tops[k] = s_all.top[k * 32 + lane];
        R.m = fmaxf(R.m, tops[k]);
    }
    R.m = warp_max(R.m);
    if (R.m == -INFINITY) {  // nothing is left to choose from
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            a.logprob[row] = -INFINITY;
        }
        return;
    }
    // Tokens from x0 on are listed. The least of the 32 largest logits of as many parts of the row has 32 tokens from it on and
    // about 130 where they lie anywhere, the k-th largest of the 128 maxima at least k. A list that turns out too short
    // or too long is not used.
    float x0 = R.m;
    const bool infinite = R.m == INFINITY;
    if (infinite) {  // the infinite logits share everything
        R.mine = -INFINITY;
        for (int v = v0 + lane; v < v1; v += 32) {
            T* x = reinterpret_cast<T*>(s_data + v);
            for (int e = 0; e < VE; ++e) {
                const bool top = (float)x[e] == INFINITY;
                x[e] = value_of<T>(top ? 0.f : -INFINITY);
                if (top) R.mine = 0.f;
            }
        }
        R.m = x0 = 0.f;
    } else if (!greedy && cuts) {
        uint32_t key;
        if (!by_k || top_k <= 32) {
            uint32_t best = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) best = max(best, order_key(__float_as_uint(tops[k])));
            key = __reduce_min_sync(0xffffffffu, best);
        } else {
            // each of 128 threads finds its maximum's place among all of them
            if (tid < kParts) {
                const float y = s_all.top[tid];
                int ahead = 0;
                for (int i = 0; i < kParts; i += 4) {
                    const float4 z = *reinterpret_cast<const float4*>(s_all.top + i);
                    ahead += (z.x > y || (z.x == y && i < tid)) + (z.y > y || (z.y == y && i + 1 < tid)) +
                             (z.z > y || (z.z == y && i + 2 < tid)) + (z.w > y || (z.w == y && i + 3 < tid));
                }
                if (ahead == imin(top_k, kParts - 8) - 1) s_found[0] = order_key(__float_as_uint(y));
            }
            __syncthreads();
            key = (uint32_t)s_found[0];
        }
        x0 = __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
        x0 = x0 == x0 ? fminf(x0, R.m) : -INFINITY;  // (few groups have anything: the key is below that of -infinity)
        if (by_min && !by_k && !by_p)  // a little below what min-p keeps
            x0 = fmaxf(x0, R.m + T_ * __logf(fminf(min_p, 1.f)) - fabsf(R.m) * 0x1p-10f - T_ * 0x1p-6f);
        if (!(x0 > -INFINITY)) x0 = -3.402823466e38f;
    }

    // ---- sums of the quick weights, at T = 1 for the log-probability and, where they are asked for, at T
    const bool quick = !greedy && !by_k && (by_p || !by_min);
    const bool two = quick && temp != 1.f;
    u64 quick_z = 0, whole_z = 0;
    List& list = s_work.list;
    uint2* to = cl.map_shared_rank(&s_work, 0)->list.raw + rank * (kList / a.ctas);
    for (int turn = 0;; ++turn) {
        const float half_m = 0.5f * R.m, c1 = -2.8853900817779268f;
        float s1 = 0.f, st = 0.f;
        float mine = 0.f;  // weight of what this thread has listed
        int largest = 0;
        for (int v = v0 + lane; v < v1; v += 32) {
            const uint4 raw = s_data[v];
            float x[VE];
            float2 y = make_float2(0.f, 0.f), yt = y;
            unpack<T>(raw, x);
#pragma unroll
            for (int e = 0; e < VE; e += 2) {
                const float2 h = tc::fma2(make_float2(x[e], x[e + 1]), make_float2(-0.5f, -0.5f), make_float2(half_m, half_m));
                const float2 t1 = tc::mul2(h, make_float2(c1, c1));
                y = tc::add2(y, make_float2(ex2(t1.x), ex2(t1.y)));
                if (two) {
                    const float2 tt = tc::mul2(h, make_float2(R.c2, R.c2));
                    yt = tc::add2(yt, make_float2(ex2(tt.x), ex2(tt.y)));
                }
            }
            const float top = top_of<T>(raw);
            if (top == R.m) {  // the largest weigh 1 and are counted, so that the sum of the others keeps its own precision
                y = yt = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float h = fmaf(-0.5f, x[e], half_m);
                    if (x[e] == R.m) ++largest;
                    y.x += x[e] == R.m ? 0.f : ex2(h * c1);
                    if (two) yt.x += x[e] == R.m ? 0.f : ex2(h * R.c2);
                }
            }
            s1 += y.x + y.y;
            st += yt.x + yt.y;
            if (cuts && top >= x0) {
                unsigned hits = 0;
#pragma unroll
                for (int e = 0; e < VE; ++e) hits |= x[e] >= x0 ? 1u << e : 0u;
                int i = atomicAdd(&s_n, __popc(hits));
                for (; hits; hits &= hits - 1, ++i) {
                    const int e = __ffs(hits) - 1;
                    const float z = (float)reinterpret_cast<const T*>(s_data + v)[e];
                    mine += ex2(fmaf(-0.5f, z, half_m) * R.c2);
                    if (i < kList / a.ctas) to[i] = make_uint2(order_key(__float_as_uint(z)), (uint32_t)(first + v * VE + e - skew));
                }
            }
        }
        const bool nan = s1 != s1;
        const u64 ones = (u64)largest << kFrac;
        const u64 w1 = warp_sum(ones + (nan ? 0ull : (u64)__float2ull_rn(s1 * 0x1p44f)));
        const u64 wt = two ? warp_sum(ones + (u64)__float2ull_rn(st * 0x1p44f)) : w1;
        if (!cuts) R.tell(cl, s_all.quick, wt);
        const float wl = cuts ? warp_sum(mine) : 0.f;
        if (lane == 0) {
            s_part[0][warp] = w1;
            s_part[1][warp] = wt;
            s_part[2][warp] = __float2ull_rn(wl * 0x1p44f);
        }
        if (nan) s_nan = 1;
        __syncthreads();
        if (tid < 3 * a.ctas) {  // three sums for each CTA
            const int what = tid % 3;
            All* o = cl.map_shared_rank(&s_all, tid / 3);
            u64 s = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += s_part[what][w];
            o->sums[rank][what] = s_nan ? ~0ull : s;
            if (what == 0) {
                o->n[rank] = s_n;
                o->done[rank] = 0;
            }
        }
        cl.sync();
        whole_z = quick_z = 0;
        bool bad = false;
        for (int r = 0; r < a.ctas; ++r) {
            bad = bad || s_all.sums[r][0] == ~0ull;
            whole_z += s_all.sums[r][0];
            quick_z += s_all.sums[r][1];
        }
        if (!bad) break;
        // a NaN counts as a logit of -infinity
        for (int v = v0 + lane; v < v1; v += 32) {
            T* x = reinterpret_cast<T*>(s_data + v);
            for (int e = 0; e < VE; ++e)
                if ((float)x[e] != (float)x[e]) x[e] = value_of<T>(-INFINITY);
        }
        cl.sync();
        if (tid == 0) {
            s_n = s_nan = 0;
        }
        __syncthreads();
    }
    const u64 off = (u64)((float)quick_z * (float)kQuick) + 1;
    const u64 least_w = by_min ? mul_ceil(fminf(min_p, 1.f), 1ull << kFrac) : 0;  // min-p keeps weights from here on

    int token = -1;
    float at = 0.f;
    bool mine = false;  // this thread has the token
    // ---- the list, if all that may be kept is in it
    bool listed = cuts;
    int ln = 0;
    if (cuts) {
        u64 lw = 0;
        for (int r = 0; r < a.ctas; ++r) {
            listed = listed && s_all.n[r] <= kList / a.ctas;
            ln += s_all.n[r];
            lw += s_all.sums[r][2];
        }
        // What min-p keeps is all in the list. That is enough unless top-p goes by what the first k weigh together: min-p drops
        // some of those only afterwards, so the list has to have all k, or every token above -infinity.
        const bool by_min_all = by_min && R.exact(x0) < least_w && (!(by_k && by_p) || x0 == -3.402823466e38f);
        if (!greedy)
            // (a thread may have added up as many as 72 of the listed weights, 72 * 2^-24 = 4.3e-6: twice kQuick covers that)
            listed = listed && (by_min_all || (by_k ? ln >= top_k : by_p && lw >= mul_ceil(p, quick_z + off) + 2 * off));
    }
    if (listed) {
        if (rank != 0) return;
        u64 me = 0, w = 0;
        if (tid < ln) {
            int i = tid, r = 0;
            for (; i >= s_all.n[r]; ++r) i -= s_all.n[r];
            const uint2 y = list.raw[r * (kList / a.ctas) + i];
            list.tokens[tid] = make_ulonglong2((u64)y.x << 32 | ~y.y, R.exact(__uint_as_float(y.x & 0x80000000u ? y.x ^ 0x80000000u : ~y.x)));
        }
        __syncthreads();
        // G threads for each token, each looks at every G-th other
        int G = 1;
        while (2 * G * ln <= kThreads && G < 32) G *= 2;
        const int i = tid / G, g = tid % G;
        u64 before = 0;
        int ahead = 0;
        if (i < ln) {
            me = list.tokens[i].x;
            w = list.tokens[i].y;
#pragma unroll 4
            for (int j = g; j < ln; j += G) {
                const ulonglong2 o = list.tokens[j];
                before += o.x > me ? o.y : 0;
                ahead += o.x > me;
            }
        }
        for (int o = 1; o < G; o *= 2) {
            before += __shfl_xor_sync(0xffffffffu, before, o);
            ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
        }
        bool keep = i < ln && (greedy ? ahead == 0 : !by_k || ahead < top_k);
        if (by_p) {
            u64 lo, hi;
            if (by_k) {
                lo = hi = mul_ceil(p, R.cta_sum(keep && g == 0 ? w : 0));
            } else {
                lo = mul_ceil(p, quick_z - off);
                hi = mul_ceil(p, quick_z + off);
                if (__syncthreads_or(keep && ahead > 0 && before >= lo && before < hi)) {
                    // the sum of all weights exactly, from the row itself: the other CTAs are gone
                    const T* x = static_cast<const T*>(a.x) + (long long)row * a.stride;
                    u64 s = 0;
                    for (int j = tid; j < a.vocab; j += kThreads) {
                        float y = (float)x[j];
                        if (infinite) y = y == INFINITY ? 0.f : -INFINITY;
                        if (y > -INFINITY && j != a.barred) s += R.exact(y);
                    }
                    lo = hi = mul_ceil(p, R.cta_sum(s));
                }
            }
            keep = keep && (ahead == 0 || before < lo);
        }
        if (by_min) keep = keep && w >= least_w;
        // the kept ones, and of each the weight of those up to its number
        if (tid == 0) s_n = 0;
        const u64 all = R.cta_sum(keep && g == 0 ? w : 0);  // (its barriers order s_n)
        if (keep && g == 0) list.kept[atomicAdd(&s_n, 1)] = make_ulonglong2(me, w);
        __syncthreads();
        const int kn = s_n;
        u64 target = mul_floor(u, all), upto = 0;
        target = target < all ? target : all - 1;
        G = 1;
        while (2 * G * kn <= kThreads && G < 32) G *= 2;
        const int ki = tid / G;
        if (ki < kn) {
            me = list.kept[ki].x;
            w = list.kept[ki].y;
#pragma unroll 4
            for (int j = tid % G; j < kn; j += G) {
                const ulonglong2 o = list.kept[j];
                upto += (uint32_t)o.x >= (uint32_t)me ? o.y : 0;
            }
        }
        for (int o = 1; o < G; o *= 2) upto += __shfl_xor_sync(0xffffffffu, upto, o);
        if (ki < kn && tid % G == 0 && upto > target && upto - w <= target) {
            const uint32_t k = (uint32_t)(me >> 32);
            token = (int)~(uint32_t)me;
            at = __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
            mine = true;
        }
    } else {
        // ---- the whole row
        bool found = false;
        uint32_t cut = 0;  // kept: tokens above this key, and the first `ties` at it
        long long ties = 0;
        if (!cuts) {
            // all tokens, by quick weights
            const u64 target = mul_floor(u, quick_z);
            u64 y[kPer], s4 = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = lane * kPer + k;
                y[k] = i < a.ctas * kWarps ? s_all.quick[i] : 0;
                s4 += y[k];
            }
            const u64 upto = warp_scan(s4);
            const unsigned hit = __ballot_sync(0xffffffffu, upto > target);
            int who = -1;
            u64 base = 0;
            if (hit) {
                u64 run = upto - s4;
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    if (who < 0 && run + y[k] > target) {
                        who = lane * kPer + k;
                        base = run;
                    }
                    run += y[k];
                }
                who = __shfl_sync(0xffffffffu, who, __ffs(hit) - 1);
                base = __shfl_sync(0xffffffffu, base, __ffs(hit) - 1);
            }
            if (who >= 0 && who == rank * kWarps + warp) {
                // The error of a sum up to a token less u times all of it: each weight's counts (1 - u)-fold before the token,
                // u-fold behind it, so 2 u (1 - u) of the bound for all. The log2(n / Z) of sums of u and 1 - u of Z are larger by
                // log2(1 / u) and log2(1 / (1 - u)), which come to 6.6e-8 Z at most: a 64th of the bound covers it
                const u64 slack = (u64)((float)off * 2.f * u * (1.f - u)) + (off >> 6) + 64;
                mine = R.template walk<false>(-INFINITY, 0, 0, base, target, slack, &token, &at);
                if (mine)
                    for (int r = 0; r < a.ctas; ++r) cl.map_shared_rank(&s_all, r)->done[rank] = 1;
            }
            cl.sync();
            found = __any_sync(0xffffffffu, lane < a.ctas && s_all.done[lane]);
        }
        bool valued = false;  // the token is found from counted values
        if constexpr (sizeof(T) == 2 && Type<T>::SHIFT == 16) {
            if (!found && !greedy && R.count_values(cl)) {
                valued = true;
                Cut by{kValues, 0, 0, 0, -INFINITY};
                u64 z = s_upto.sum_weight[kThreads];
                if (by_k && s_upto.sum_count[kThreads] > top_k) {  // (masked tokens are not counted)
                    by = R.template cut_values<COUNT>(cl, (u64)top_k);
                    z = by.above + (u64)by.ties * by.w;
                }
                if (by_p) by = R.template cut_values<MASS>(cl, mul_ceil(p, z));
                if (by_min) {
                    const float x = R.at_key(R.key_from(least_w));
                    if (x > by.x) by = Cut{R.place_from(x), 1ll << 40, R.exact(x), 0, x};
                }
                // the CTA in which the sum passes u times all of it: it alone goes on. Lane r has CTA r's
                int tied;
                u64 have = R.kept_of(cl, by, &tied);
                cl.sync();  // nothing of another CTA is read from here on
                const int upto_tied = warp_scan(tied);
                const long long rest = by.ties - (upto_tied - tied);
                int allowed = rest <= 0 ? 0 : rest < tied ? (int)rest : tied;
                have += (u64)allowed * by.w;
                const u64 in = warp_scan(have), sum = __shfl_sync(0xffffffffu, in, 31);
                u64 target = mul_floor(u, sum);
                target = target < sum ? target : sum - 1;
                const int who = __ffs(__ballot_sync(0xffffffffu, in > target)) - 1;
                target -= __shfl_sync(0xffffffffu, in - have, who);
                allowed = __shfl_sync(0xffffffffu, allowed, who);
                have = __shfl_sync(0xffffffffu, have, who);
                if (who != rank) return;
                if (tid == 0) s_n = 0;
                const int below = imax(0, kFrac - 63 + __clzll(have));  // factors of two by which its sum is below 1
                const u64 slack = (u64)((float)have * ((float)kPart + below * (float)kPartOctave)) + (1ull << 15);
                // its warps' parts and the token, by quick weights and, where their error leaves it open, by exact ones
                for (int exact = 0; exact < 2; ++exact) {
                    u64 s;
                    int n;
                    if (exact) R.template kept_here<true>(by.x, &s, &n);
                    else R.template kept_here<false>(by.x, &s, &n);
                    __syncthreads();
                    if (lane == 0) {
                        s_scan[warp] = s;
                        s_all.ties[warp] = n;
                    }
                    __syncthreads();
                    const int at_warp = lane < kWarps ? s_all.ties[lane] : 0, left = allowed - (warp_scan(at_warp) - at_warp);
                    const int count = imax(0, imin(left, at_warp));
                    const u64 y = lane < kWarps ? s_scan[lane] + (u64)count * by.w : 0, upto = warp_scan(y);
                    const unsigned hit = __ballot_sync(0xffffffffu, upto > target);
                    if (hit) {
                        const int l = __ffs(hit) - 1, mine_ = __shfl_sync(0xffffffffu, count, l);
                        const u64 from = __shfl_sync(0xffffffffu, upto - y, l);
                        if (warp == l) {
                            if (exact) mine = R.template walk<true>(by.x, mine_, by.w, from, target, 0, &token, &at);
                            else mine = R.template walk<false>(by.x, mine_, by.w, from, target, slack, &token, &at);
                            if (mine) s_n = 1;
                        }
                    }
                    __syncthreads();
                    if (s_n) break;
                }
            }
        }
        if (found || valued) {
        } else if (!cuts) {
            R.weigh(cl, cut, false);
        } else if (greedy) {
            cut = R.key_of(R.m);
            ties = 1;
            R.weigh(cl, cut, false);
        } else {
            uint32_t key_k = 0;
            long long ties_k = 0;
            u64 skipped;
            if (by_k) {
                cut = key_k = R.template select<COUNT>(cl, (u64)top_k, -INFINITY, &skipped);
                ties = ties_k = top_k - (long long)skipped;
                R.weigh(cl, cut, false);
            }
            if (by_p) {
                u64 z = quick_z;
                if (by_k) {
                    const long long have = R.total_ties();
                    z = R.total(s_all.quick) + (u64)(have < ties_k ? have : ties_k) * R.exact(R.at_key(key_k));
                }
                cut = R.template select<MASS>(cl, mul_ceil(p, z), by_k ? R.at_key(key_k) : -INFINITY, &skipped);
                // From quick weights that key is the right one or near it; exact ones tell. The next keys are tried first. Where
                // single tokens weigh much less than the quick sums are off by, the cut lies thousands of tokens away: then steps grow
                // fourfold until they pass it, and what is known of it is halved (fewer than 50 times in all).
                uint32_t lo = by_k ? key_k - 1 : R.key_of(-INFINITY), hi = R.key_of(R.m) + 1;  // lo < the cut's key < hi
                for (int turn = 0;; ++turn) {
                    R.weigh(cl, cut, !by_k);
                    const u64 above = R.total(s_all.quick), w = R.exact(R.at_key(cut));
                    long long have = R.total_ties();
                    if (!by_k) z = above + (u64)have * w + R.total(s_all.whole);
                    else if (cut == key_k) have = have < ties_k ? have : ties_k;
                    const u64 target = mul_ceil(p, z);
                    if (above < target && above + (u64)have * w >= target) {
                        ties = (long long)((target - above + w - 1) / w);
                        break;
                    }
                    const bool up = above >= target;
                    if (up) lo = cut;
                    else hi = cut;
                    if (turn < 3) {
                        cut = R.next_key(cl, cut, up);
                    } else {
                        const uint32_t half = (hi - lo) / 2, step = min(1u << 2 * min(turn - 2, 15), half);
                        cut = up ? lo + step : hi - step;
                    }
                }
            }
            if (by_min) {
                const uint32_t k = R.key_from(least_w);
                if (k > cut) {
                    cut = k;
                    ties = 1ll << 40;
                    R.weigh(cl, cut, false);
                }
            }
        }
        if (!found && !valued) {
            // what each warp's part keeps, and the part in which the sum passes u times all of it
            const u64 tie_w = ties ? R.exact(R.at_key(cut)) : 0;
            int have[kPer], take[kPer], n4 = 0;
            u64 y[kPer], s4 = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = lane * kPer + k;
                have[k] = i < a.ctas * kWarps ? s_all.ties[i] : 0;
                n4 += have[k];
            }
            long long rest = ties - (warp_scan(n4) - n4);
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = lane * kPer + k;
                take[k] = rest <= 0 ? 0 : rest < have[k] ? (int)rest : have[k];
                rest -= have[k];
                y[k] = i < a.ctas * kWarps ? s_all.quick[i] + (u64)take[k] * tie_w : 0;
                s4 += y[k];
            }
            const u64 upto = warp_scan(s4), all = __shfl_sync(0xffffffffu, upto, 31);
            u64 target = mul_floor(u, all);
            target = target < all ? target : all - 1;  // (the largest logit weighs something, so all > 0)
            const int l = __ffs(__ballot_sync(0xffffffffu, upto > target)) - 1;
            int who = -1, allowed = 0;
            u64 run = upto - s4, base = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                if (who < 0 && run + y[k] > target) {
                    who = lane * kPer + k;
                    base = run;
                    allowed = take[k];
                }
                run += y[k];
            }
            who = __shfl_sync(0xffffffffu, who, l);
            base = __shfl_sync(0xffffffffu, base, l);
            allowed = __shfl_sync(0xffffffffu, allowed, l);
            if (who == rank * kWarps + warp)
                mine = R.template walk<true>(cut ? R.at_key(cut) : -INFINITY, allowed, tie_w, base, target, 0, &token, &at);
        }
        token += first - skew;
    }
    if (mine) {
        // whole_z is at least 1; near it the logarithm is taken of what it is more
        constexpr u64 one = 1ull << kFrac;
        const float lz = whole_z < 2 * one ? log1pf((float)(whole_z > one ? whole_z - one : 0) * 0x1p-44f) : logf((float)whole_z * 0x1p-44f);
        a.token[row] = token;
        // at - m - lz, the two sums with their errors (Knuth), so that it is rounded once
        const float d = BDLM_ADD(at, -R.m), db = BDLM_ADD(d, -at), s = BDLM_ADD(d, -lz), sb = BDLM_ADD(s, -d);
        const float de = BDLM_ADD(BDLM_ADD(at, -BDLM_ADD(d, -db)), BDLM_ADD(-R.m, -db)), se = BDLM_ADD(BDLM_ADD(d, -BDLM_ADD(s, -sb)), BDLM_ADD(-lz, -sb));
        a.logprob[row] = BDLM_ADD(s, BDLM_ADD(de, se));
    }
}

template <typename T>
cudaError_t launch(SampleArgs a, int num_sms, cudaStream_t st, int* launches) {
    constexpr int VE = Type<T>::VE;
    // A CTA's part of a row: at most 64 KB, so that two CTAs share an SM; parts of a lone row may be smaller, so that
    // more SMs take part, but a warp should have a vector for each lane.
    auto parts = [&](int c) { return ((a.vocab + c - 1) / c + 63) / 64 * 64; };
    int c = 1;
    while (c < kMaxCtas && (size_t)parts(c) * sizeof(T) > 65536) c *= 2;
    while (c < kMaxCtas && (long long)a.rows * c * 2 <= num_sms && parts(c) > kThreads * VE) c *= 2;
    a.ctas = c;
    a.per = parts(c);
    a.ahead = 2 * num_sms / c * c;  // two CTAs on an SM
    const size_t smem = ((size_t)a.per / VE + 1) * 16;
    // (what the longest row needs, whatever this one does: calls of several threads set the same)
    constexpr int most = kMaxVocab / kMaxCtas * (int)sizeof(T) + 16;
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
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
