// sample.cuh - the weights of tokens, and what the sampling kernel is given.
//
// A token's weight is w = e^((x - m) / T) with the row's largest logit m. Two
// forms of it are used. The quick one is a multiplication and an exponential of
// the special-function unit. Its errors, 2^-22 of the exponential, the roundings
// of the argument and those of the sums, move any sum of weights of a row by
// less than kQuick of the row's sum Z. An argument t = -log2 w is half the
// distance times 2 log2(e) / T: three roundings and the constant's own, a fifth
// of one, so it is off by at most 3.2 |t| 2^-24. The sum of w |t| over n tokens
// is at most Z log2(n / Z), and Z >= 1: 18 * 3.2 * 2^-24 * ln 2 = 2.4e-6. The
// exponential adds 2.4e-7, and at most 20 additions in 32 bits 20 * 2^-24 =
// 1.2e-6, together 3.9e-6.
//
// A sum z over one CTA's part of a row (of counted values: at most 2^15 tokens
// of 16 bits, nine vectors of a thread and so 37 additions) may be far below 1: 15
// + log2(1 / z) take the place of 18. With 2.4e-7 and 37 * 2^-24 that is 4.5e-6 z
// and 1.33e-7 z for each factor of two by which z is below 1. Sums of whole multiples of 2^-44 are off by up to
// half a unit for each of 2^15 tokens (the exact ones leave out what is below
// 2^-45) and 2^10 partial sums, less than 2^15 units.
//
// The exact one is a whole multiple of 2^-44, from two-float arithmetic (sums
// and products with their errors after Dekker and Knuth; a table of 2^(j/16)
// and the series of e^y). Its relative error is below 2^-40, sums of it are
// sums of integers, the same in any order, and equal logits weigh the same.
#pragma once

#include <cstdint>

#include <cmath>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace bdlm {
namespace sample {

constexpr double kQuick = 4e-6, kPart = 4.6e-6, kPartOctave = 1.4e-7;
constexpr int kMaxVocab = 1 << 18;
constexpr int kFrac = 44;  // a weight of 1 is 2^44: 2^18 of them stay below 2^62

#ifdef __CUDA_ARCH__
#define BDLM_MUL(a, b) __fmul_rn(a, b)
#define BDLM_ADD(a, b) __fadd_rn(a, b)
#define BDLM_FMA(a, b, c) __fmaf_rn(a, b, c)
#define BDLM_RINT(x) __float2int_rn(x)
#else
#define BDLM_MUL(a, b) ((a) * (b))
#define BDLM_ADD(a, b) ((a) + (b))
#define BDLM_FMA(a, b, c) std::fma(a, b, c)
#define BDLM_RINT(x) ((int)std::lrint(x))
#endif

struct F2 {
    float hi, lo;
};

// 2^(j / 16), j = -8 .. 8, as two floats each.
constexpr int kTable = 17;
#define BDLM_POW2_TABLE                                                                                                      \
    {0x1.6a09e6p-1f, 0x1.9fcef4p-27f}, {0x1.7a1148p-1f, -0x1.829fd0p-26f}, {0x1.8ace54p-1f, 0x1.15506ep-28f},                \
        {0x1.9c4918p-1f, 0x1.51f848p-28f}, {0x1.ae89fap-1f, -0x1.a94b14p-27f}, {0x1.c199bep-1f, -0x1.3d56b2p-28f},           \
        {0x1.d5818ep-1f, -0x1.822dbcp-28f}, {0x1.ea4afap-1f, 0x1.52486cp-28f}, {1.f, 0.f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f}, \
        {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.306fe0p+0f, 0x1.4636e2p-25f},            \
        {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},           \
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}

// 2^44 e^((x - m) / T), rounded; c = 2 log2(e) / T. Halves of x and m are taken, so that no difference overflows.
__host__ __device__ __forceinline__ uint64_t exact_weight(float x, float m, F2 c, const F2* table) {
    const float a = BDLM_MUL(0.5f, m), b = BDLM_MUL(-0.5f, x);
    const float h = BDLM_ADD(a, b);  // half the distance, with its error
    const float bb = BDLM_ADD(h, -a);
    const float hl = BDLM_ADD(BDLM_ADD(a, -BDLM_ADD(h, -bb)), BDLM_ADD(b, -bb));
    const float th = BDLM_MUL(h, c.hi);
    if (!(th < 46.f && th > -1.f)) return 0;  // below half of 2^-44 (and x = -inf); logits above m have no weight
    const float tl = BDLM_ADD(BDLM_FMA(h, c.hi, -th), BDLM_FMA(h, c.lo, BDLM_MUL(hl, c.hi)));
    const int n = BDLM_RINT(th);
    const float f = BDLM_ADD((float)n, -th);  // exact; the weight is 2^-n 2^(f - tl)
    const int j = BDLM_RINT(BDLM_MUL(f, 16.f));
    const float r = BDLM_FMA((float)j, -0.0625f, f);  // exact
    constexpr float lh = 0x1.62e430p-1f, ll = -0x1.05c610p-29f;  // ln 2
    const float y0 = BDLM_MUL(r, lh), y1 = BDLM_ADD(BDLM_FMA(r, lh, -y0), BDLM_FMA(r, ll, BDLM_MUL(-lh, tl)));
    const float yh = BDLM_ADD(y0, y1), yl = BDLM_ADD(y1, -BDLM_ADD(yh, -y0));
    const float qh = BDLM_MUL(yh, yh), ql = BDLM_FMA(BDLM_MUL(2.f, yh), yl, BDLM_FMA(yh, yh, -qh));
    float p = BDLM_FMA(yh, 1.f / 720.f, 1.f / 120.f);
    p = BDLM_FMA(yh, p, 1.f / 24.f);
    p = BDLM_FMA(yh, p, 1.f / 6.f);
    const float sh = BDLM_FMA(0.5f, qh, yh), se = BDLM_FMA(0.5f, qh, -BDLM_ADD(sh, -yh));
    const float low = BDLM_ADD(BDLM_FMA(BDLM_MUL(qh, yh), p, se), BDLM_FMA(0.5f, ql, yl));
    const F2 t = table[j + 8];
    const float ph = BDLM_MUL(t.hi, sh), pl = BDLM_FMA(t.hi, sh, -ph);
    const float rh = BDLM_ADD(t.hi, ph), re = BDLM_ADD(ph, -BDLM_ADD(rh, -t.hi));
    const float rl = BDLM_ADD(BDLM_ADD(re, pl), BDLM_ADD(t.lo, BDLM_FMA(t.hi, low, BDLM_MUL(t.lo, sh))));
    // rh is a multiple of 2^-25
    const int64_t w = ((int64_t)BDLM_RINT(BDLM_MUL(rh, 0x1p25f)) << (kFrac - 25)) + BDLM_RINT(BDLM_MUL(rl, 0x1p44f));
    return (uint64_t)((2 * w + ((int64_t)1 << n)) >> (n + 1));
}

#ifdef __CUDACC__
// Two of them at once: the same steps on pairs (two operations per instruction), the roundings of n and j to whole
// numbers by adding and taking off 1.5 * 2^23.
__device__ __forceinline__ void exact_weights(float x0, float x1, float m, F2 c, const F2* table, unsigned long long& w0,
                                              unsigned long long& w1) {
    using tc::add2;
    using tc::fma2;
    using tc::mul2;
    auto two = [](float v) { return make_float2(v, v); };
    auto less = [&](float2 u, float2 v) { return fma2(v, two(-1.f), u); };  // u - v (a negated operand would cost two more)
    constexpr float whole = 12582912.f, lh = 0x1.62e430p-1f, ll = -0x1.05c610p-29f;
    const float2 a = two(0.5f * m), b = mul2(two(-0.5f), make_float2(x0, x1));
    const float2 h = add2(a, b), bb = less(h, a);
    const float2 hl = add2(less(a, less(h, bb)), less(b, bb));
    const float2 th = mul2(h, two(c.hi));
    const float2 tm = mul2(h, two(-c.hi));  // -th
    const float2 tl = add2(fma2(h, two(c.hi), tm), fma2(h, two(c.lo), mul2(hl, two(c.hi))));
    const float2 nw = add2(th, two(whole)), f = add2(add2(nw, two(-whole)), tm);
    const float2 jw = fma2(f, two(16.f), two(whole)), r = fma2(add2(jw, two(-whole)), two(-0.0625f), f);
    const float2 y0 = mul2(r, two(lh)), ym = mul2(r, two(-lh));
    const float2 y1 = add2(fma2(r, two(lh), ym), fma2(r, two(ll), mul2(two(-lh), tl)));
    const float2 yh = add2(y0, y1), yl = less(y1, less(yh, y0));
    const float2 qh = mul2(yh, yh), ql = fma2(mul2(two(2.f), yh), yl, fma2(yh, yh, mul2(qh, two(-1.f))));
    float2 p = fma2(yh, two(1.f / 720.f), two(1.f / 120.f));
    p = fma2(yh, p, two(1.f / 24.f));
    p = fma2(yh, p, two(1.f / 6.f));
    const float2 sh = fma2(two(0.5f), qh, yh), se = fma2(two(0.5f), qh, less(yh, sh));
    const float2 low = add2(fma2(mul2(qh, yh), p, se), fma2(two(0.5f), ql, yl));
    const bool some0 = th.x < 46.f && th.x > -1.f, some1 = th.y < 46.f && th.y > -1.f;
    const F2 t0 = table[some0 ? __float_as_int(jw.x) - 0x4b400000 + 8 : 0], t1 = table[some1 ? __float_as_int(jw.y) - 0x4b400000 + 8 : 0];
    const float2 ht = make_float2(t0.hi, t1.hi), lt = make_float2(t0.lo, t1.lo);
    const float2 ph = mul2(ht, sh), pl = fma2(ht, sh, mul2(ph, two(-1.f)));
    const float2 rh = add2(ht, ph), re = less(ph, less(rh, ht));
    const float2 rl = add2(add2(re, pl), add2(lt, fma2(ht, low, mul2(lt, sh))));
    const float2 big = mul2(rh, two(0x1p25f)), small = mul2(rl, two(0x1p44f));
    auto join = [](float hi, float lo, float nw) {
        const int n = (__float_as_int(nw) - 0x4b400000) & 63;
        const int64_t w = ((int64_t)__float2int_rn(hi) << (kFrac - 25)) + __float2int_rn(lo);
        return (uint64_t)((2 * w + ((int64_t)1 << n)) >> (n + 1));
    };
    w0 = some0 ? join(big.x, small.x, nw.x) : 0;
    w1 = some1 ? join(big.y, small.y, nw.y) : 0;
}
#endif

// A key that orders floats as their values do; -0 and 0 have the same.
__host__ __device__ __forceinline__ uint32_t order_key(uint32_t bits) {
    if (bits == 0x80000000u) bits = 0;
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

}  // namespace sample

// What a call samples with: per-row arrays, or where they are null one value for all rows.
struct SampleArgs {
    const void* x;  // logits: row i begins at element i * stride
    long long stride;
    int rows, vocab;
    const float* u;
    const float* temperature;
    const int* top_k;
    const float* top_p;
    const float* min_p;
    float temperature_all, top_p_all, min_p_all;
    int top_k_all;
    const int* now;  // rows whose entry is not `want` are left (nullptr: none are)
    int want;
    int barred;  // token without weight (-1: none)
    int* token;
    float* logprob;
    int ctas;  // CTAs of a row, one cluster
    int per;    // elements of each
    int ahead;  // CTAs that run at a time, whole clusters
};
cudaError_t launch_sample(SampleArgs a, int dtype, int num_sms, cudaStream_t st, int* launches);

struct UnmaskArgs {
    const int* now;
    const int* sampled;
    const float* logprob;
    const int* cu_rows;
    int n_seqs, total_rows, mask_id;
    const int* n_min;
    const float* threshold;
    int n_min_all;
    float threshold_all;
    int* out;
    int* left;
    WsHeader* hdr;
};
cudaError_t launch_unmask(const UnmaskArgs& a, cudaStream_t st, int* launches);

}  // namespace bdlm
