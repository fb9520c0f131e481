// cache_merge.cuh - joins the partial results of the attention over the paged
// cache (cache_attn.cuh says how the work is cut).
//
// The merge has kSlices CTAs per boundary between two shares. The CTAs whose
// boundaries fall into one unit take equal runs of its rows, read the rows of
// all its partials (a warp's 32 rows are 512 consecutive bytes of every float4
// column) and write o and lse. What they read has just been written, so it is
// bound by the latency of L2: the weights of a CTA's rows are worked out once,
// in shared memory, and the partials of a row are asked for four at a time. It
// is launched with programmatic dependence: its CTAs come up as the
// attention's leave, and wait for its memory. From the last share's
// end to the call's takes 4 us for one token, 15 for 152 partials of 256 rows
// (20 MB).
#pragma once

#include <cuda_fp16.h>

#include "cache_attn.cuh"
#include "tc_ptx.cuh"

namespace bdlm {
namespace {

using namespace cattn;

constexpr int kMergeThreads = 256;
// 64 rows over 131072 keys (152 partials of 256 rows), whole call: 140, 139, 140, 147, 157 us with 1, 2, 3, 4, 8 slices;
// 37 short ragged sequences 41.4, 40.3, 38.5, 38.3, 38.9.
constexpr int kSlices = 3;
constexpr int kMaxParts = kMaxCtas + 1;

// (four CTAs to an SM: the compiler takes 79 registers for d = 64 unless it is told, and a short call then 1.3 us more of 13)
template <int D, bool RUNS>
__global__ void __launch_bounds__(kMergeThreads, D == 64 ? 4 : 0) cache_merge_kernel(const CacheAttnArgs a, int ctas) {
    __shared__ float s_w[kMaxParts][32];  // weights of 32 rows at a time
    __shared__ float s_lse[32];
    __shared__ int s_err[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (RUNS) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const ShareRec* recs = share_recs(a.scratch);
    const int c = blockIdx.x + 1;
    if (blockIdx.x == 0 && blockIdx.y == 0) {  // the shares' errors
        int err = 0, info = 0;
        for (int i = tid; i < ctas; i += kMergeThreads)
            if (recs[i].error) {
                err = recs[i].error;
                info = recs[i].info;
            }
        if (tid == 0) s_err[0] = s_err[1] = 0;
        __syncthreads();
        if (err && atomicCAS(&s_err[0], 0, err) == 0) s_err[1] = info;
        __syncthreads();
        if (tid == 0) {
            a.hdr->error = s_err[0];
            a.hdr->info = s_err[1];
        }
    }
    if (c >= ctas) return;  // a single CTA: it leaves one record and cuts nothing
    const ShareRec r = recs[c];
    const int rows = imin(unit_rows<RUNS>(), r.rows * a.G - r.m0), two = RUNS ? 0 : is_two(rows), lead = lead_of(rows);
    if (c >= r.C || tile_at(r.off, two, lead) == 0) return;  // no share begins here, or it begins with its unit's first tile
    auto begin = [&](int i) { return share_begin(r.per, r.more, i); };
    const long long g0 = begin(c) - r.off;
    int c0 = c, c1 = c;  // boundaries inside the unit: shares c0 - 1 .. c1 hold its partials
    while (c0 > 1 && begin(c0 - 1) > g0 && tile_at((int)(begin(c0 - 1) - g0), two, lead) > 0) --c0;
    while (c1 + 1 < r.C && begin(c1 + 1) < g0 + r.cost) ++c1;
    const int parts = c1 - c0 + 2;
    const int slices = (c1 - c0 + 1) * kSlices, slice = (c - c0) * kSlices + blockIdx.y;
    const int lo = rows * slice / slices, hi = rows * (slice + 1) / slices;
    const int R = slot_rows(a.total_rows, a.G);
    const bool plane = RUNS && r.part != PART_WHOLE;
    auto slot = [&](int p) { return slot_at(a.scratch, p == 0 ? 2 * (c0 - 1) + 1 : 2 * (c0 - 1 + p), R, D); };
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int n = imin(32, hi - i0);
        // one warp per partial: a lane's row's lse
        for (int p = warp; p < parts; p += kMergeThreads / 32)
            if (lane < n) s_w[p][lane] = __ldcg(slot(p) + (long long)R * D + i0 + lane);
        __syncthreads();
        if (warp == 0 && lane < n) {
            float mx = -INFINITY, z = 0.f;
            bool nan = false;
            for (int p = 0; p < parts; ++p) {
                const float x = s_w[p][lane];
                mx = fmaxf(mx, x);
                nan = nan || x != x;
            }
            for (int p = 0; p < parts; ++p) {
                const float x = s_w[p][lane], w = exp2f(x - mx);
                s_w[p][lane] = x == -INFINITY ? -1.f : w;
                if (x != -INFINITY) z += w;
            }
            const float inv = nan ? NAN : z > 0.f ? 1.f / z : 0.f;
            // -1: the row sees no key of the partial, which is not read; a weight of 0 is (it may hold NaN)
            for (int p = 0; p < parts; ++p) s_w[p][lane] = s_w[p][lane] < 0.f ? -1.f : s_w[p][lane] * inv;
            s_lse[lane] = nan ? NAN : z > 0.f ? mx + log2f(z) : -INFINITY;  // base 2
        }
        __syncthreads();
        // item: eight columns of one row; consecutive threads take consecutive rows
        for (int it = tid; it < 32 * (D / 8); it += kMergeThreads) {
            const int k = it & 31, q = it >> 5;
            if (k >= n) continue;
            float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int p0 = 0; p0 < parts; p0 += 4) {
                float4 v[4][2];
                float w[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    w[u] = p0 + u < parts ? s_w[p0 + u][k] : -1.f;
                    if (!(w[u] < 0.f)) {
                        const float4* s = reinterpret_cast<const float4*>(slot(p0 + u)) + (long long)(2 * q) * R + i0 + k;
                        v[u][0] = __ldcg(s);
                        v[u][1] = __ldcg(s + R);
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (!(w[u] < 0.f)) {
                        const float y[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w, v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = fmaf(w[u], y[e], o[e]);
                    }
            }
            const int m = r.m0 + i0 + k, row = r.row0 + m / a.G, h = r.head * a.G + m % a.G;
            if (plane) {
                const long long flat = a.plane_rows, to = (long long)r.row0 + m;
                float4* dst = reinterpret_cast<float4*>(plane_o(a, D, r.part, r.head)) + 2 * q * flat + to;
                dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                dst[flat] = make_float4(o[4], o[5], o[6], o[7]);
                if (q == 0) plane_lse(a, D, r.part, r.head)[to] = s_lse[k];
                continue;
            }
            const long long at = ((long long)row * a.H + h) * D + 8 * q;
            if (a.o_f32) {
                *reinterpret_cast<float4*>(a.o_f32 + at) = make_float4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<float4*>(a.o_f32 + at + 4) = make_float4(o[4], o[5], o[6], o[7]);
            } else {
                uint32_t b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 y = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
                    b[e] = *reinterpret_cast<const uint32_t*>(&y);
                }
                *reinterpret_cast<uint4*>(a.o + at) = make_uint4(b[0], b[1], b[2], b[3]);
            }
            if (q == 0) a.lse[(long long)h * a.total_rows + row] = s_lse[k] * 0.69314718055994531f;
        }
        __syncthreads();
    }
}

template <bool RUNS>
cudaError_t launch_merge(const CacheAttnArgs& a, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ctas > 1 ? ctas - 1 : 1), kSlices);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return a.c.D == 128 ? cudaLaunchKernelEx(&cfg, cache_merge_kernel<128, RUNS>, a, ctas)
                        : cudaLaunchKernelEx(&cfg, cache_merge_kernel<64, RUNS>, a, ctas);
}

}  // namespace
}  // namespace bdlm
