// cache_attn_shared.cu - launches the attention in which what a run of
// sequences shares is read once (cache_attn.cuh), and does what is left of it.
#include "cache_merge.cuh"

namespace bdlm {
namespace {

// What is left of a call with runs, for one sequence and kv head:
//   few rows, few keys  the rows' attention over the keys that the sequence has of its own, joined with what its run shares;
//   else                the two planes of a run's rows joined; nothing for a sequence that reads alone.
//
// The first has no use for tiles of 128 flat rows: one token has G of them, and a unit of the kernel with such tiles takes 10 us
// to begin and to end. Here MMAs have the flat rows, at most 8, as their short side: S = K Q^T and O^T = V^T P^T, 16 keys or 16
// columns by 8 rows by 16, on fp16 operands. e4m3 codes are exact in fp16. A row of Q is scaled by a power of two that
// puts its largest between 2^14 and 2^15, so that entries down to 2^-31 of that stay exact (bf16 has 8 bits) and a smaller
// one loses at most 2^-39 of it. Weights, scaled by 2^15, are two fp16 terms: each is off by at most 2^-23 of itself or 2^-40.
// Sums are fp32; the scales are applied to sums of 16 keys, which lie in one page.
// Each warp takes 16 keys at a time, with a running maximum of its own, and copies them to shared memory three times ahead; the
// warps' results are joined at the end. The order of columns within Q and K, and of columns of V, is the one in which a
// lane's operands lie side by side in a key's row; vectors of a row change places with its number, so that 8 lanes meet no bank
// twice. Bound by latency for short ones (the table, the first keys, the joins), by memory for long ones: 64 rows over up to
// 1024 own keys of 8 heads, 57 MB, take 28 us with cold caches (43 with products in fp32 instead of MMAs), 256 over 4096, 2.1 GB, about
// 340.
//
// The second has a warp read eight rows' float4 of four pairs of columns, runs of 128 bytes, and write runs of 64.
constexpr int kOwnThreads = 256;
constexpr int kOwnStages = 3;
template <int D>
constexpr int own_smem() { return kOwnThreads / 32 * kOwnStages * 2 * 16 * D; }

__device__ __forceinline__ float ex2o(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two e4m3 codes -> fp16; four, the first two and the last two
__device__ __forceinline__ void widen4(uint32_t c, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(c));
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // of an 8 x 8 matrix of fp16 across the warp
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
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
__device__ __forceinline__ void join_planes(const CacheAttnArgs& a, const SeqRows& q, int plane, int head) {
    constexpr int CG = D / 32;  // groups of four pairs of float4
    const int lane = threadIdx.x & 31, groups = (q.rows * a.G + 7) / 8, each = kOwnThreads / 32;
    const long long flat = a.plane_rows;
    for (int it = blockIdx.z * each + (threadIdx.x >> 5); it < groups * CG; it += gridDim.z * each) {
        const int c = it % CG * 4 + (lane >> 3), m = it / CG * 8 + (lane & 7);  // eight columns from 8 c on of flat row m
        if (m >= q.rows * a.G) continue;
        const long long at = (long long)plane + m;
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
    // V: 16-byte vectors of a key. A lane has 16 T columns of a key in the first product, W of a value in the second.
    constexpr int WARPS = kOwnThreads / 32, V = D / 16, T = D / 64, W = D / 8, LOADS = D / 32, R = kFewRows;
    static_assert(R == 8, "the short side of an MMA");
    static_assert(kMostKeys <= 16 * 32 * WARPS, "one page of 16 keys per lane");
    static_assert(WARPS * R * D * 4 <= own_smem<D>(), "the warps' results take the place of keys");
    extern __shared__ uint4 s_ring[];  // [WARPS][kOwnStages][16 keys, 16 values][V]; in the end O of each warp, [WARPS][R][D]
    __shared__ float s_top[WARPS][R], s_sum[WARPS][R];
    const int s = blockIdx.x, head = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const SeqRows q = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s);
    const Run run = run_of<true, true>(a, s, q, nullptr);  // (malformed ones must not be followed)
    const bool few = q.ok && run.ok && q.rows > 0 && is_few(a, q.rows, q.len - run.shared);
    if (!few) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (!share_recs(a.scratch)[0].bad && q.rows > 0 && run.shared > 0) join_planes<D>(a, q, run.plane, head);
        return;
    }
    if (blockIdx.z > 0) return;
    const int flat = q.rows * a.G, key0 = run.shared, g = lane >> 2, t = lane & 3;
    auto end_of = [&](int m) { return key_end(q.len, a.block, q.pos0 + imin(m, flat - 1) / a.G) - key0; };  // keys (from key0 on) that it sees
    const int most = end_of(flat - 1), least = end_of(0), end0 = end_of(2 * t), end1 = end_of(2 * t + 1);
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
    uint4* ring = s_ring + warp * kOwnStages * 32 * V;
    auto place = [](int key, int v) { return key * V + (v ^ (D == 128 ? key & 7 : key >> 1 & 3)); };
    // Copies the i-th 16 keys of this warp and their values. Always a group, so that counting them is enough.
    auto copy = [&](int i) {
        if (i < n) {
            const long long page = __shfl_sync(0xffffffffu, id, i);
            const int row = (key0 + 16 * (warp + WARPS * i)) & (a.c.page - 1);
            const long long from = ((page * a.c.Hk + head) * a.c.page + row) * D;
            uint4* to = ring + i % kOwnStages * 32 * V;
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const int at = 32 * j + lane, x = place(at / V, at % V);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_addr(to + x)), "l"(a.c.k + from + 16 * at) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_addr(to + 16 * V + x)), "l"(a.c.v + from + 16 * at) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kOwnStages; ++i) copy(i);

    // ---- this lane's columns of row g, 16 T from 16 T t on, as fp16
    uint32_t qf[4 * T][2];
    float unscale0, unscale1;  // rows 2 t and 2 t + 1
    {
        const int m = imin(g, flat - 1);
        const uint4* src = reinterpret_cast<const uint4*>(a.q + ((long long)(q.row0 + m / a.G) * a.H + head * a.G + m % a.G) * D + 16 * T * t);
        alignas(16) uint32_t w[8 * T];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * T; ++j) *reinterpret_cast<uint4*>(w + 4 * j) = __ldg(src + j);
#pragma unroll
        for (int j = 0; j < 8 * T; ++j)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e <= top < 2^(e + 1): scaled by 2^(14 - e). From e = -100 down a smaller factor does, and infinity stays what it is.
        const int e = imin(imax((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
        const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23), down = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
        for (int j = 0; j < 8 * T; ++j) qf[j / 2][j & 1] = half2_of(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
        unscale0 = __shfl_sync(0xffffffffu, down, 8 * t);
        unscale1 = __shfl_sync(0xffffffffu, down, 8 * t + 4);
    }
    float top0 = -INFINITY, top1 = -INFINITY, sum0 = 0.f, sum1 = 0.f;  // of the rows 2 t and 2 t + 1, as o's pairs
    float2 o[W];  // columns W g + i
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = make_float2(0.f, 0.f);
    for (int i = 0; i < n; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kOwnStages - 1) : "memory");
        __syncwarp();
        const uint4* keys = ring + i % kOwnStages * 32 * V;
        const int first = 16 * (warp + WARPS * i);
        float x[4] = {0.f, 0.f, 0.f, 0.f};  // keys g and g + 8, rows 2 t and 2 t + 1 of each
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const uint4 y0 = keys[place(g, T * t + j)], y1 = keys[place(g + 8, T * t + j)];
            const uint32_t w0[4] = {y0.x, y0.y, y0.z, y0.w}, w1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t a0, a1, a2, a3;
                widen4(w0[k], a0, a2);
                widen4(w1[k], a1, a3);
                mma(x, a0, a1, a2, a3, qf[4 * j + k][0], qf[4 * j + k][1]);
            }
        }
        const float scale = a.scale_log2 * __shfl_sync(0xffffffffu, ks, i), vscale = __shfl_sync(0xffffffffu, vs, i) * 0x1p-15f;
        x[0] = first + g < end0 ? x[0] * unscale0 * scale : -INFINITY;
        x[1] = first + g < end1 ? x[1] * unscale1 * scale : -INFINITY;
        x[2] = first + g + 8 < end0 ? x[2] * unscale0 * scale : -INFINITY;
        x[3] = first + g + 8 < end1 ? x[3] * unscale1 * scale : -INFINITY;
        float new0 = fmaxf(x[0], x[2]), new1 = fmaxf(x[1], x[3]);
#pragma unroll
        for (int k = 4; k < 32; k *= 2) {
            new0 = fmaxf(new0, __shfl_xor_sync(0xffffffffu, new0, k));
            new1 = fmaxf(new1, __shfl_xor_sync(0xffffffffu, new1, k));
        }
        new0 = fmaxf(new0, top0);
        new1 = fmaxf(new1, top1);
        // (a row that sees no key yet has weights e^(-inf - 0) = 0)
        const float from0 = new0 == -INFINITY ? 0.f : new0, from1 = new1 == -INFINITY ? 0.f : new1;
        const float2 less = make_float2(ex2o(top0 - from0), ex2o(top1 - from1));
        top0 = new0;
        top1 = new1;
        x[0] = ex2o(x[0] - from0);
        x[1] = ex2o(x[1] - from1);
        x[2] = ex2o(x[2] - from0);
        x[3] = ex2o(x[3] - from1);
        sum0 = fmaf(sum0, less.x, x[0] + x[2]);
        sum1 = fmaf(sum1, less.y, x[1] + x[3]);
#pragma unroll
        for (int k = 0; k < W; ++k) o[k] = tc::mul2(o[k], less);
        uint32_t hi[2], lo[2];  // keys 2 t, 2 t + 1 (and 8 more) of row g
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float p0 = x[2 * k] * 0x1p15f, p1 = x[2 * k + 1] * 0x1p15f;
            const uint32_t h = half2_of(p0, p1);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            hi[k] = transposed(h);
            lo[k] = transposed(half2_of(p0 - f.x, p1 - f.y));
        }
        // ---- values. Rows that see different numbers of these keys take turns, with the values that they do not see taken as 0:
        // what a masked key holds reaches no row
        const int in0 = imin(imax(end0 - first, 0), 16), in1 = imin(imax(end1 - first, 0), 16);
        for (int in = imin(imax(least - first, 0), 16);;) {
            if (in > 0) {
                const uint4* values = keys + 16 * V;
                alignas(16) uint32_t y[4][W / 4];  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9; columns W g ..
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int key = 2 * t + (k & 1) + (k & 2) * 4;
                    if constexpr (D == 128) {
                        *reinterpret_cast<uint4*>(y[k]) = values[place(key, g)];
                    } else {
                        *reinterpret_cast<uint2*>(y[k]) = *(reinterpret_cast<const uint2*>(values + place(key, g >> 1)) + (g & 1));
                    }
                    if (key >= in)
#pragma unroll
                        for (int e = 0; e < W / 4; ++e) y[k][e] = 0;
                }
                const bool take0 = in0 == in, take1 = in1 == in;
                const float2 by = make_float2(take0 ? vscale : 0.f, take1 ? vscale : 0.f);
#pragma unroll
                for (int e = 0; e < W / 4; ++e)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // two columns of two keys each
                        const uint32_t c0 = __byte_perm(y[0][e], y[1][e], h ? 0x7362 : 0x5140), c1 = __byte_perm(y[2][e], y[3][e], h ? 0x7362 : 0x5140);
                        uint32_t a0, a1, a2, a3;
                        float z[4] = {0.f, 0.f, 0.f, 0.f};
                        widen4(c0, a0, a1);
                        widen4(c1, a2, a3);
                        mma(z, a0, a1, a2, a3, hi[0], hi[1]);
                        mma(z, a0, a1, a2, a3, lo[0], lo[1]);
                        // (a NaN of rows whose turn it is not)
                        z[0] = take0 ? z[0] : 0.f;
                        z[1] = take1 ? z[1] : 0.f;
                        z[2] = take0 ? z[2] : 0.f;
                        z[3] = take1 ? z[3] : 0.f;
                        const int col = 4 * e + 2 * h;
                        o[col] = tc::fma2(make_float2(z[0], z[1]), by, o[col]);
                        o[col + 1] = tc::fma2(make_float2(z[2], z[3]), by, o[col + 1]);
                    }
            }
            in = (int)__reduce_min_sync(0xffffffffu, (unsigned)imin(in0 > in ? in0 : 99, in1 > in ? in1 : 99));
            if (in > 16) break;
        }
        __syncwarp();  // all lanes have read the stage
        copy(i + kOwnStages);
    }
#pragma unroll
    for (int k = 4; k < 32; k *= 2) {
        sum0 += __shfl_xor_sync(0xffffffffu, sum0, k);
        sum1 += __shfl_xor_sync(0xffffffffu, sum1, k);
    }
    if (g == 0) {
        s_top[warp][2 * t] = top0;
        s_top[warp][2 * t + 1] = top1;
        s_sum[warp][2 * t] = sum0;
        s_sum[warp][2 * t + 1] = sum1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // the keys are used up
    float* s_o = reinterpret_cast<float*>(s_ring);
#pragma unroll
    for (int i = 0; i < W; i += 4) {
        float* to = s_o + (warp * R + 2 * t) * D + W * g + i;
        *reinterpret_cast<float4*>(to) = make_float4(o[i].x, o[i + 1].x, o[i + 2].x, o[i + 3].x);
        *reinterpret_cast<float4*>(to + D) = make_float4(o[i].y, o[i + 1].y, o[i + 2].y, o[i + 3].y);
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what the run shares, and the error word
    if (share_recs(a.scratch)[0].bad) return;
    if (bad) set_error(a.hdr, DEV_CHECK, s);
    const long long all = a.plane_rows;
    for (int it = tid; it < flat * (D / 8); it += kOwnThreads) {
        const int m = it / (D / 8), c = it % (D / 8);
        float top = -INFINITY, z = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, w0 = 0.f, l0 = -INFINITY;
        float4 x0 = make_float4(0.f, 0.f, 0.f, 0.f), x1 = x0;
        if (key0 > 0) {
            const long long at = (long long)run.plane + m;
            l0 = __ldcg(plane_lse(a, D, PART_SHARED, head) + at);
            const float4* p0 = reinterpret_cast<const float4*>(plane_o(a, D, PART_SHARED, head)) + 2 * c * all + at;
            x0 = __ldcg(p0);
            x1 = __ldcg(p0 + all);
            top = l0;
        }
        bool nan = l0 != l0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_top[w][m]);
        const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float by = ex2o(s_top[w][m] - from);
            const float4* p = reinterpret_cast<const float4*>(s_o + (w * R + m) * D + 8 * c);
            const float4 v0 = p[0], v1 = p[1];
            const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            z = fmaf(s_sum[w][m], by, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(v[e], by, y[e]);
        }
        if (key0 > 0) {
            w0 = ex2o(l0 - from);
            z += w0;
            const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(x[e], w0, y[e]);
        }
        nan = nan || z != z;
        const float inv = nan ? NAN : z > 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= inv;
        const int row = q.row0 + m / a.G, h = head * a.G + m % a.G;
        put_row<D>(a, row, h, c, y);
        if (c == 0) a.lse[(long long)h * a.total_rows + row] = nan ? NAN : z > 0.f ? (top + log2f(z)) * 0.69314718055994531f : -INFINITY;
    }
}

}  // namespace

long long cache_attn_plane_rows(long long total_rows, int G, int n_seqs) {
    const long long flat = total_rows * G, most = (long long)kPlaneRows * n_seqs;
    return flat < most ? flat : most;
}
size_t cache_attn_plane_bytes(long long plane_rows, int Hk, int D) {
    return (sizeof(float) * 2 * (size_t)plane_rows * Hk * (D + 1) + 255) / 256 * 256;
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
