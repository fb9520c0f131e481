// cache_attn_shared.cu - launches the attention in which what a run of
// sequences shares is read once (cache_attn.cuh), and does what is left of it.
#include "cache_merge.cuh"

namespace bdlm {
namespace {

// What is left of a call with runs, for one sequence and kv head:
//   few rows, few keys  the rows' attention over the keys that the sequence has of its own, joined with what its run shares;
//   else                the two planes of a run's rows joined; nothing for a sequence that reads alone.
//
// The first has no use for MMA tiles: one token has G flat rows of 128, and a unit of the tensor-core kernel takes 10 us
// to begin and to end. It is done by multiplying in fp32, four flat rows at a time, in three steps: the scores
// of all keys into shared memory, D / 16 lanes to a key, 16 columns each; their softmax; and the weighted sum of the values, in
// which each such group of lanes has sums of its own over the keys that it meets. Each warp takes 16 keys at a time,
// which lie in one page; a lane copies what it will read of them to shared memory, four times ahead, keys first and then
// values. Bound by latency: of the table, of the first keys, of the joins.
//
// The second has a warp read eight rows' float4 of four pairs of columns, runs of 128 bytes, and write runs of 64.
constexpr int kOwnThreads = 256;
constexpr int kOwnRows = 4;
constexpr int kOwnStages = 4;
template <int D>
constexpr int own_smem() { return kOwnThreads / 32 * kOwnStages * 16 * D + kOwnRows * kFewKeys * 4; }

__device__ __forceinline__ float ex2o(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// four e4m3 codes -> floats
__device__ __forceinline__ void widen4(uint32_t c, float* f) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(c));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = x.x;
    f[1] = x.y;
    f[2] = y.x;
    f[3] = y.y;
}

template <int D>
__device__ __forceinline__ void put_row(const CacheAttnArgs& a, int row, int h, int c, const float (&o)[8]) {  // columns 8 c ..
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
}

template <int D>
__device__ __forceinline__ void join_planes(const CacheAttnArgs& a, const SeqRows& q, int head) {
    constexpr int CG = D / 32;  // groups of four pairs of float4
    const int lane = threadIdx.x & 31, groups = (q.rows * a.G + 7) / 8, each = kOwnThreads / 32;
    const long long flat = (long long)a.total_rows * a.G;
    for (int it = blockIdx.z * each + (threadIdx.x >> 5); it < groups * CG; it += gridDim.z * each) {
        const int c = it % CG * 4 + (lane >> 3), m = it / CG * 8 + (lane & 7);  // eight columns from 8 c on of flat row m
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
        put_row<D>(a, row, h, c, o);
        if (c == 0) a.lse[(long long)h * a.total_rows + row] = nan ? NAN : z > 0.f ? (mx + log2f(z)) * 0.69314718055994531f : -INFINITY;
    }
}

template <int D>
__global__ void __launch_bounds__(kOwnThreads, 2) cache_own_kernel(const CacheAttnArgs a) {
    constexpr int LPK = D / 16, KPI = 32 / LPK, LOADS = 16 / KPI, WARPS = kOwnThreads / 32, R = kOwnRows;
    static_assert(kFewKeys <= 16 * 32 * WARPS, "one page of 16 keys per lane");
    static_assert(WARPS * D <= kFewKeys && WARPS == 2 * R, "sums take the place of scores; two warps have a row's softmax");
    extern __shared__ uint4 s_ring[];  // [WARPS][kOwnStages][LOADS][32]
    // scores, then weights; in the end O of each warp, [WARPS][R][D]
    float(*s_p)[kFewKeys] = reinterpret_cast<float(*)[kFewKeys]>(s_ring + WARPS * kOwnStages * LOADS * 32);
    __shared__ float s_top[WARPS], s_sum[WARPS];
    const int s = blockIdx.x, head = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const SeqRows q = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s);
    const Run run = run_of<true>(a, s, q);  // (malformed ones must not be followed)
    const bool few = q.ok && run.ok && q.rows > 0 && is_few(a, q.rows, q.len - run.shared);
    if (!few) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (!share_recs(a.scratch)[0].bad && q.rows > 0 && run.shared > 0) join_planes<D>(a, q, head);
        return;
    }
    if (blockIdx.z > 0) return;
    const int flat = q.rows * a.G, key0 = run.shared, slice = lane % LPK, mine = lane / LPK;
    const int most = key_end(q.len, a.block, q.pos0 + q.rows - 1) - key0;  // keys (from key0 on) that the last row sees
    // lane i has the page and scales of the i-th 16 keys of this warp
    const int chunks = (most + 15) / 16, n = chunks > warp ? (chunks - warp + WARPS - 1) / WARPS : 0;
    int id = 0;
    float ks = 0.f, vs = 0.f;
    bool bad = false;
    if (lane < n) {
        id = __ldg(a.c.table + (long long)s * a.c.max_pages + ((key0 + 16 * (warp + WARPS * lane)) >> a.c.page_shift));
        bad = id < 0 || id >= a.c.n_pages;
        if (bad) id = 0;  // some page of the pool stands in, and its scale makes the rows that see it NaN
        ks = bad ? NAN : __ldg(a.c.k_scale + (long long)id * a.c.Hk + head);
        vs = __ldg(a.c.v_scale + (long long)id * a.c.Hk + head);
    }
    uint4* ring = s_ring + warp * kOwnStages * LOADS * 32 + lane;
    // Copies the i-th 16 keys of this warp, or from n on the (i - n)-th 16 values. Always a group, so that counting them is enough.
    auto copy = [&](int i) {
        if (i < 2 * n) {
            const int c = i < n ? i : i - n;
            const long long page = __shfl_sync(0xffffffffu, id, c);
            const int row = (key0 + 16 * (warp + WARPS * c)) & (a.c.page - 1);
            const uint8_t* at = (i < n ? a.c.k : a.c.v) + ((page * a.c.Hk + head) * a.c.page + row) * D + 16 * lane;
            const uint32_t to = tc::smem_addr(ring + i % kOwnStages * LOADS * 32);
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512 * j), "l"(at + 512 * j) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto wait = [] { asm volatile("cp.async.wait_group %0;" ::"n"(kOwnStages - 1) : "memory"); };
    auto widen16 = [](const uint4& y, float (&x)[16]) {
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) widen4(w[e], x + 4 * e);
    };
    const long long all = (long long)a.total_rows * a.G;
    for (int m0 = 0; m0 < flat; m0 += R) {
        int end[R];  // keys that the rows see
#pragma unroll
        for (int f = 0; f < R; ++f) end[f] = key_end(q.len, a.block, q.pos0 + imin(m0 + f, flat - 1) / a.G) - key0;
#pragma unroll
        for (int i = 0; i < kOwnStages; ++i) copy(i);
        {  // ---- scores
            float2 qf[R][8];  // this lane's 16 columns of the rows
#pragma unroll
            for (int f = 0; f < R; ++f) {
                const int m = imin(m0 + f, flat - 1);
                const uint4* src = reinterpret_cast<const uint4*>(a.q + ((long long)(q.row0 + m / a.G) * a.H + head * a.G + m % a.G) * D + 16 * slice);
                const uint4 u[2] = {__ldg(src), __ldg(src + 1)};
                const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) qf[f][e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
            }
            for (int i = 0; i < n; ++i) {
                wait();
                const float scale = a.scale_log2 * __shfl_sync(0xffffffffu, ks, i);
                const uint4* k = ring + i % kOwnStages * LOADS * 32;
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    float x[16], dot[R];
                    widen16(k[32 * j], x);
#pragma unroll
                    for (int f = 0; f < R; ++f) {
                        float2 t = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) t = tc::fma2(qf[f][e], make_float2(x[2 * e], x[2 * e + 1]), t);
                        dot[f] = t.x + t.y;
                    }
                    // a lane ends up with one row's sum: half of the rows go to the lane across, and half of those again
                    const bool up = slice & (LPK / 2), left = slice & (LPK / 4);
                    const float v0 = (up ? dot[2] : dot[0]) + __shfl_xor_sync(0xffffffffu, up ? dot[0] : dot[2], LPK / 2);
                    const float v1 = (up ? dot[3] : dot[1]) + __shfl_xor_sync(0xffffffffu, up ? dot[1] : dot[3], LPK / 2);
                    float y = (left ? v1 : v0) + __shfl_xor_sync(0xffffffffu, left ? v0 : v1, LPK / 4);
                    if (LPK == 8) y += __shfl_xor_sync(0xffffffffu, y, 1);
                    const int key = 16 * (warp + WARPS * i) + KPI * j + mine, sees = up ? (left ? end[3] : end[2]) : left ? end[1] : end[0];
                    if (LPK == 4 || !(slice & 1)) s_p[(up ? 2 : 0) + (left ? 1 : 0)][key] = key < sees ? y * scale : -INFINITY;
                }
                copy(i + kOwnStages);
            }
        }
        __syncthreads();
        {  // ---- softmax: two warps to a row
            float* p = s_p[warp >> 1];
            float top = -INFINITY, sum = 0.f;
            bool nan = false;
            for (int i = (warp & 1) * 32 + lane; i < 16 * chunks; i += 64) {
                top = fmaxf(top, p[i]);
                nan = nan || p[i] != p[i];
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (__any_sync(0xffffffffu, nan)) top = NAN;
            if (lane == 0) s_top[warp] = top;
            __syncthreads();
            const float other = s_top[warp ^ 1];
            top = top != top || other != other ? NAN : fmaxf(top, other);
            for (int i = (warp & 1) * 32 + lane; i < 16 * chunks; i += 64) {
                const float y = top == -INFINITY ? 0.f : ex2o(p[i] - top);
                p[i] = y;
                sum += y;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            __syncthreads();  // both have read the other's
            if (lane == 0) {
                s_top[warp] = top;
                s_sum[warp] = sum;
            }
        }
        __syncthreads();
        float2 o[R][8];
#pragma unroll
        for (int f = 0; f < R; ++f)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[f][e] = make_float2(0.f, 0.f);
        for (int i = 0; i < n; ++i) {  // ---- values
            wait();
            const float scale = __shfl_sync(0xffffffffu, vs, i);
            const uint4* v = ring + (n + i) % kOwnStages * LOADS * 32;
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const int key = 16 * (warp + WARPS * i) + KPI * j + mine;
                float x[16];
                widen16(v[32 * j], x);
#pragma unroll
                for (int f = 0; f < R; ++f) {
                    if (key >= end[f]) continue;  // what a masked key holds reaches no row
                    const float w = s_p[f][key] * scale;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[f][e] = tc::fma2(make_float2(w, w), make_float2(x[2 * e], x[2 * e + 1]), o[f][e]);
                }
            }
            copy(n + i + kOwnStages);
        }
        __syncthreads();  // the weights are used up
        float* s_o = &s_p[0][0];
#pragma unroll
        for (int f = 0; f < R; ++f)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float2 y = o[f][e];
#pragma unroll
                for (int x = LPK; x < 32; x *= 2) {
                    y.x += __shfl_xor_sync(0xffffffffu, y.x, x);
                    y.y += __shfl_xor_sync(0xffffffffu, y.y, x);
                }
                if (mine == 0) *reinterpret_cast<float2*>(s_o + (warp * R + f) * D + 16 * slice + 2 * e) = y;
            }
        __syncthreads();
        if (m0 == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");  // what the run shares, and the error word
            if (share_recs(a.scratch)[0].bad) return;
            if (bad) set_error(a.hdr, DEV_CHECK, s);
        }
        for (int it = tid; it < R * (D / 8); it += kOwnThreads) {
            const int f = it / (D / 8), c = it % (D / 8), m = m0 + f;
            if (m >= flat) continue;
            float top = s_top[2 * f], z = s_sum[2 * f] + s_sum[2 * f + 1], y[8];
            bool nan = top != top;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) y[e] += s_o[(w * R + f) * D + 8 * c + e];
            }
            if (key0 > 0) {
                const long long at = (long long)q.row0 * a.G + m;
                const float l0 = __ldcg(plane_lse(a, D, PART_SHARED, head) + at);
                const float4* p0 = reinterpret_cast<const float4*>(plane_o(a, D, PART_SHARED, head)) + 2 * c * all + at;
                const float4 x0 = __ldcg(p0), x1 = __ldcg(p0 + all);
                const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                nan = nan || l0 != l0;
                const float both = fmaxf(top, l0), w0 = l0 == -INFINITY ? 0.f : ex2o(l0 - both), w1 = top == -INFINITY ? 0.f : ex2o(top - both);
                z = fmaf(z, w1, w0);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], w1, x[e] * w0);
                top = both;
            }
            const float inv = nan ? NAN : z > 0.f ? 1.f / z : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= inv;
            const int row = q.row0 + m / a.G, h = head * a.G + m % a.G;
            put_row<D>(a, row, h, c, y);
            if (c == 0) a.lse[(long long)h * a.total_rows + row] = nan ? NAN : z > 0.f ? (top + log2f(z)) * 0.69314718055994531f : -INFINITY;
        }
        __syncthreads();  // the next rows' scores take the place of these sums
    }
}

}  // namespace

size_t cache_attn_plane_bytes(long long total_rows, int H, int D) {
    return (sizeof(float) * 2 * (size_t)total_rows * H * (D + 1) + 255) / 256 * 256;
}

cudaError_t launch_cache_attn_shared(const CacheAttnArgs& a, int num_sms, cudaStream_t st, int* launches) {
    const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    cudaError_t e = a.c.D == 128 ? launch_cache_attn_runs_d128(a, ctas, st) : launch_cache_attn_runs_d64(a, ctas, st);
    if (e == cudaSuccess) e = launch_merge<true>(a, ctas, st);
    if (e != cudaSuccess) return e;
    // slices of a join
    const long long pairs = (long long)a.c.n_seqs * a.c.Hk, fill = (3LL * num_sms + pairs - 1) / pairs;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.c.n_seqs, (unsigned)a.c.Hk, (unsigned)(fill > 64 ? 64 : fill));
    cfg.blockDim = dim3(kOwnThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    auto own = [&](auto kernel, int smem) {
        cfg.dynamicSmemBytes = smem;
        const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return err != cudaSuccess ? err : cudaLaunchKernelEx(&cfg, kernel, a);
    };
    e = a.c.D == 128 ? own(cache_own_kernel<128>, own_smem<128>()) : own(cache_own_kernel<64>, own_smem<64>());
    if (e == cudaSuccess) *launches += 3;
    return e;
}

}  // namespace bdlm
