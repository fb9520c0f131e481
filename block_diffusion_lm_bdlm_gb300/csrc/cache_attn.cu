// cache_attn.cu - attention of new rows over the paged 8-bit cache.
//
// One CTA per (row, query head): the keys that the row sees pass in chunks of
// 128, one key per thread for the scores, one column per thread for the
// weighted sum of the values, with the running maximum and sum of an online
// softmax in fp32.
#include "cache.cuh"

namespace bdlm {
namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(256) check_kernel(const CacheAttnArgs a) {
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0x7fffffff;
    __syncthreads();
    for (int s = threadIdx.x; s < a.c.n_seqs; s += 256)
        if (!seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s).ok) atomicMin(&s_bad, s);
    __syncthreads();
    if (threadIdx.x == 0) {
        a.hdr->error = s_bad == 0x7fffffff ? DEV_OK : DEV_CHECK;
        a.hdr->info = s_bad == 0x7fffffff ? 0 : s_bad;
        a.hdr->counter = s_bad != 0x7fffffff;  // nothing is written
    }
}

__device__ __forceinline__ float code_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

__device__ float block_max(float x, float* buf) {
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    x = fmaxf(fmaxf(buf[0], buf[1]), fmaxf(buf[2], buf[3]));
    __syncthreads();
    return x;
}
__device__ float block_sum(float x, float* buf) {
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    x = buf[0] + buf[1] + (buf[2] + buf[3]);
    __syncthreads();
    return x;
}

__global__ void __launch_bounds__(kThreads) simple_kernel(const CacheAttnArgs a) {
    __shared__ float s_q[128], s_p[kThreads], buf[4];
    __shared__ int s_bad;
    const CacheView& c = a.c;
    if (a.hdr->counter) return;
    const int row = blockIdx.x, h = blockIdx.y, kh = h / a.G, tid = threadIdx.x, D = c.D;
    if (tid == 0) s_bad = 0;
    if (row >= __ldg(a.cu_rows + c.n_seqs)) return;
    int lo = 0, hi = c.n_seqs;  // the last sequence with cu_rows[s] <= row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu_rows + mid) <= row) lo = mid; else hi = mid;
    }
    const SeqRows r = seq_rows(c, a.cu_rows, a.q_pos, a.total_rows, lo);
    const int end = key_end(r.len, a.block, r.pos0 + row - r.row0);
    const int* pages = c.table + (long long)lo * c.max_pages;
    if (tid < D) s_q[tid] = __bfloat162float(a.q[((long long)row * a.H + h) * D + tid]);
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int k0 = 0; k0 < end; k0 += kThreads) {
        float x = -INFINITY;
        const int j = k0 + tid;
        if (j < end) {
            const int id = __ldg(pages + (j >> c.page_shift));
            if (id < 0 || id >= c.n_pages) {
                s_bad = 1;
            } else {
                const long long unit = (long long)id * c.Hk + kh;
                const uint4* k = reinterpret_cast<const uint4*>(c.k + (unit * c.page + (j & (c.page - 1))) * D);
                float dot = 0.f;
                for (int e = 0; e < D / 16; ++e) {
                    const uint4 u = __ldg(k + e);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                    for (int b = 0; b < 16; ++b)
                        dot = fmaf(s_q[16 * e + b], code_value((uint8_t)(w[b >> 2] >> (8 * (b & 3)))), dot);
                }
                x = dot * __ldg(c.k_scale + unit) * a.scale_log2;
            }
        }
        const float big = block_max(x, buf);
        const bool nan = __syncthreads_or(x != x);
        const float m_new = nan ? NAN : fmaxf(m, big);
        const float p = j < end ? exp2f(x - m_new) : 0.f;
        const float fade = m == -INFINITY ? 0.f : exp2f(m - m_new);
        s_p[tid] = p;
        l = l * fade + block_sum(p, buf);
        acc *= fade;
        m = m_new;
        if (tid < D)
            for (int e = 0; e < kThreads && k0 + e < end; ++e) {
                const int id = __ldg(pages + ((k0 + e) >> c.page_shift));
                if (id < 0 || id >= c.n_pages) continue;
                const long long unit = (long long)id * c.Hk + kh;
                const uint8_t v = __ldg(c.v + (unit * c.page + ((k0 + e) & (c.page - 1))) * D + tid);
                acc = fmaf(s_p[e] * __ldg(c.v_scale + unit), code_value(v), acc);
            }
        __syncthreads();
    }
    float out = end > 0 ? acc / l : 0.f, lse = end > 0 ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    if (s_bad) out = lse = NAN;
    if (tid < D) {
        const long long at = ((long long)row * a.H + h) * D + tid;
        if (a.o_f32) a.o_f32[at] = out; else a.o[at] = __float2bfloat16(out);
    }
    if (tid == 0) {
        a.lse[(long long)h * a.total_rows + row] = lse;
        if (s_bad) set_error(a.hdr, DEV_CHECK, -1);
    }
}

}  // namespace

size_t cache_attn_scratch_bytes(long long, int, int, int, int) { return 256; }

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int, cudaStream_t st, int* launches) {
    check_kernel<<<1, 256, 0, st>>>(a);
    simple_kernel<<<dim3(a.total_rows, a.H), kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *launches += 2;
    return e;
}

}  // namespace bdlm
