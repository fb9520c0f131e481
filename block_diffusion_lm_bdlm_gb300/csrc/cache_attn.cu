// cache_attn.cu - launches the attention over the paged cache and joins its
// partial results (cache_attn.cuh says how the work is cut).
//
// The merge has one CTA per boundary between two shares. The CTAs whose
// boundaries fall into one unit take equal runs of its rows, read the rows of
// all its partials (a warp's 32 rows are 512 consecutive bytes of every float4
// column) and write o and lse. It is launched with programmatic dependence:
// its CTAs come up as the attention's leave, and wait for its memory.
#include "cache_attn.cuh"

namespace bdlm {
namespace {

using namespace cattn;

constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) cache_merge_kernel(const CacheAttnArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const ShareRec* recs = share_recs(a.scratch);
    const int c = blockIdx.x + 1;
    if (blockIdx.x == 0) {  // the shares' errors
        const int n = gridDim.x + 1;
        int err = 0, info = 0;
        for (int i = threadIdx.x; i < n; i += kMergeThreads)
            if (recs[i].error) {
                err = recs[i].error;
                info = recs[i].info;
            }
        __shared__ int s_err[2];
        if (threadIdx.x == 0) s_err[0] = s_err[1] = 0;
        __syncthreads();
        if (err && atomicCAS(&s_err[0], 0, err) == 0) s_err[1] = info;
        __syncthreads();
        if (threadIdx.x == 0) {
            a.hdr->error = s_err[0];
            a.hdr->info = s_err[1];
        }
    }
    const ShareRec r = recs[c];
    const int two = r.rows * a.G - r.m0 > kUnitRows / 2;
    if (c >= r.C || tile_at(r.off, two) == 0) return;  // no share begins here, or it begins with its unit's first tile
    auto begin = [&](int i) { return share_begin(r.per, r.more, i); };
    const long long g0 = begin(c) - r.off;
    int c0 = c, c1 = c;  // boundaries inside the unit: shares c0 - 1 .. c1 hold its partials
    while (c0 > 1 && begin(c0 - 1) > g0 && tile_at((int)(begin(c0 - 1) - g0), two) > 0) --c0;
    while (c1 + 1 < r.C && begin(c1 + 1) < g0 + r.cost) ++c1;
    const int rows = imin(kUnitRows, r.rows * a.G - r.m0), parts = c1 - c0 + 2;
    const int lo = rows * (c - c0) / (c1 - c0 + 1), hi = rows * (c - c0 + 1) / (c1 - c0 + 1);
    const int R = slot_rows(a.total_rows, a.G);
    auto slot = [&](int p) { return slot_at(a.scratch, p == 0 ? 2 * (c0 - 1) + 1 : 2 * (c0 - 1 + p), R, D); };
    // item: one float4 of columns of one row; consecutive threads take consecutive rows
    const int n = hi - lo;
    for (int it = threadIdx.x; it < n * (D / 4); it += kMergeThreads) {
        const int i = lo + it % n, q = it / n, m = r.m0 + i;
        float mx = -INFINITY;
        bool nan = false;
        for (int p = 0; p < parts; ++p) {
            const float x = __ldcg(slot(p) + (long long)R * D + i);
            mx = fmaxf(mx, x);
            nan = nan || x != x;
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float z = 0.f;
        for (int p = 0; p < parts; ++p) {
            const float* s = slot(p);
            const float x = __ldcg(s + (long long)R * D + i);
            if (x == -INFINITY) continue;
            const float w = exp2f(x - mx);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + (long long)q * R + i);
            z += w;
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
        }
        const float inv = nan ? NAN : z > 0.f ? 1.f / z : 0.f;
        const int row = r.row0 + m / a.G, h = r.head * a.G + m % a.G;
        const long long at = ((long long)row * a.H + h) * D + 4 * q;
        if (a.o_f32) {
            *reinterpret_cast<float4*>(a.o_f32 + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        } else {
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), b1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(a.o + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
        }
        if (q == 0) a.lse[(long long)h * a.total_rows + row] = nan ? NAN : z > 0.f ? (mx + log2f(z)) * 0.69314718055994531f : -INFINITY;
    }
}

}  // namespace

size_t cache_attn_scratch_bytes(long long total_rows, int H, int Hk, int D, int) {
    const int rows = slot_rows(total_rows, H / Hk);
    return sizeof(ShareRec) * kMaxCtas + sizeof(float) * 2 * kMaxCtas * (size_t)slot_floats(rows, D);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int num_sms, cudaStream_t st, int* launches) {
    const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    cudaError_t e = a.c.D == 128 ? launch_cache_attn_d128(a, ctas, st) : launch_cache_attn_d64(a, ctas, st);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ctas > 1 ? ctas - 1 : 1));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = a.c.D == 128 ? cudaLaunchKernelEx(&cfg, cache_merge_kernel<128>, a) : cudaLaunchKernelEx(&cfg, cache_merge_kernel<64>, a);
    if (e == cudaSuccess) *launches += 2;
    return e;
}

}  // namespace bdlm
