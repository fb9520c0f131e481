// cache_attn.cu - launches the attention over the paged cache and joins its
// partial results (cache_attn.cuh says how the work is cut).
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
#include "cache_attn.cuh"

namespace bdlm {
namespace {

using namespace cattn;

constexpr int kMergeThreads = 256;
// 64 rows over 131072 keys (152 partials of 256 rows), whole call: 140, 139, 140, 147, 157 us with 1, 2, 3, 4, 8 slices;
// 37 short ragged sequences 41.4, 40.3, 38.5, 38.3, 38.9.
constexpr int kSlices = 3;
constexpr int kMaxParts = kMaxCtas + 1;

template <int D, bool RUNS>
__global__ void __launch_bounds__(kMergeThreads) cache_merge_kernel(const CacheAttnArgs a, int ctas) {
    __shared__ float s_w[kMaxParts][32];  // weights of 32 rows at a time
    __shared__ float s_lse[32];
    __shared__ int s_err[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    const int rows = imin(kUnitRows, r.rows * a.G - r.m0), two = is_two(rows), lead = lead_of(rows);
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
                const long long flat = (long long)a.total_rows * a.G, to = (long long)r.row0 * a.G + m;
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

// Joins the two planes for the rows of runs: a thread takes eight columns of a
// flat row of a kv head. A warp reads eight rows' float4 of four pairs of columns,
// runs of 128 bytes, and writes runs of 64 (bf16). blockIdx.x is the sequence,
// blockIdx.y a run of its items. Bound by what it moves, 8 bytes a value
// read and 2 written, most of it out of L2.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const CacheAttnArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (share_recs(a.scratch)[0].bad) return;
    const int s = blockIdx.x, lane = threadIdx.x & 31;
    const SeqRows q = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s);
    if (q.rows == 0 || run_of(a, s, q).shared == 0) return;
    constexpr int CG = D / 32;  // groups of four pairs of float4
    const long long flat = (long long)a.total_rows * a.G;
    const int groups = (q.rows * a.G + 7) / 8, each = kJoinThreads / 32;
    const long long items = (long long)a.c.Hk * groups * CG;
    for (long long it = (long long)blockIdx.y * each + (threadIdx.x >> 5); it < items; it += (long long)gridDim.y * each) {
        const int cg = (int)(it % CG), c = cg * 4 + (lane >> 3);  // eight columns from 8 c on
        const int m = (int)(it / CG % groups) * 8 + (lane & 7), head = (int)(it / CG / groups);
        if (m >= q.rows * a.G) continue;
        const long long at = (long long)q.row0 * a.G + m;
        const float l0 = __ldcg(plane_lse(a, D, PART_SHARED, head) + at), l1 = __ldcg(plane_lse(a, D, PART_OWN, head) + at);
        const float4* p0 = reinterpret_cast<const float4*>(plane_o(a, D, PART_SHARED, head)) + 2 * c * flat + at;
        const float4* p1 = reinterpret_cast<const float4*>(plane_o(a, D, PART_OWN, head)) + 2 * c * flat + at;
        const float4 x0 = __ldcg(p0), x1 = __ldcg(p0 + flat), y0 = __ldcg(p1), y1 = __ldcg(p1 + flat);
        const float mx = fmaxf(l0, l1);
        const bool nan = l0 != l0 || l1 != l1;
        float w0 = l0 == -INFINITY ? 0.f : exp2f(l0 - mx), w1 = l1 == -INFINITY ? 0.f : exp2f(l1 - mx);
        const float z = w0 + w1, inv = nan ? NAN : z > 0.f ? 1.f / z : 0.f;
        w0 *= inv;
        w1 *= inv;
        const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w}, y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)  // a part that sees no key holds zeros; a weight of 0 does not hide a NaN
            o[e] = fmaf(w0, x[e], w1 * y[e]);
        const int row = q.row0 + m / a.G, h = head * a.G + m % a.G;
        const long long to = ((long long)row * a.H + h) * D + 8 * c;
        if (a.o_f32) {
            *reinterpret_cast<float4*>(a.o_f32 + to) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4*>(a.o_f32 + to + 4) = make_float4(o[4], o[5], o[6], o[7]);
        } else {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
                b[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(a.o + to) = make_uint4(b[0], b[1], b[2], b[3]);
        }
        if (c == 0) a.lse[(long long)h * a.total_rows + row] = nan ? NAN : z > 0.f ? (mx + log2f(z)) * 0.69314718055994531f : -INFINITY;
    }
}

}  // namespace

size_t cache_attn_plane_bytes(long long total_rows, int H, int D) {
    return (sizeof(float) * 2 * (size_t)total_rows * H * (D + 1) + 255) / 256 * 256;
}

size_t cache_attn_scratch_bytes(long long total_rows, int H, int Hk, int D, int) {
    const int rows = slot_rows(total_rows, H / Hk);
    return sizeof(ShareRec) * kMaxCtas + sizeof(float) * 2 * kMaxCtas * (size_t)slot_floats(rows, D);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int num_sms, cudaStream_t st, int* launches) {
    const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    cudaError_t e;
    if (a.runs)
        e = a.c.D == 128 ? launch_cache_attn_runs_d128(a, ctas, st) : launch_cache_attn_runs_d64(a, ctas, st);
    else
        e = a.c.D == 128 ? launch_cache_attn_d128(a, ctas, st) : launch_cache_attn_d64(a, ctas, st);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ctas > 1 ? ctas - 1 : 1), kSlices);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (a.runs)
        e = a.c.D == 128 ? cudaLaunchKernelEx(&cfg, cache_merge_kernel<128, true>, a, ctas)
                          : cudaLaunchKernelEx(&cfg, cache_merge_kernel<64, true>, a, ctas);
    else
        e = a.c.D == 128 ? cudaLaunchKernelEx(&cfg, cache_merge_kernel<128, false>, a, ctas)
                          : cudaLaunchKernelEx(&cfg, cache_merge_kernel<64, false>, a, ctas);
    if (e != cudaSuccess) return e;
    *launches += 2;
    if (!a.runs) return cudaSuccess;
    const int per = kJoinThreads / 32, n = a.c.n_seqs;
    const long long items = (long long)a.c.Hk * (((long long)a.total_rows * a.G + 7) / 8) * (a.c.D / 32);
    const long long most = (items + per - 1) / per, fill = (4LL * num_sms + n - 1) / n;
    cfg.gridDim = dim3((unsigned)n, (unsigned)(most < fill ? most : fill));
    cfg.blockDim = dim3(kJoinThreads);
    e = a.c.D == 128 ? cudaLaunchKernelEx(&cfg, cache_join_kernel<128>, a) : cudaLaunchKernelEx(&cfg, cache_join_kernel<64>, a);
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace bdlm
