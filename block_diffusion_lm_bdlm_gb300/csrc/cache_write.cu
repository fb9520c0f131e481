// cache_write.cu - quantises new key and value rows into the pages of the cache.
//
// One CTA takes one (touched page, kv head) of K or of V: at most page x d
// values, held in registers from their one read to their one write. Rows of
// the page before the sequence's first new row are read back (code * scale),
// the amax over both gives the new power-of-two scale (see pow2_scale), and
// every value is stored as x / s, rounded once to nearest even: the division
// by a power of two is exact, so the codes are those of the definition bit by
// bit. Kept rows are stored again only where the scale has changed.
//
// The pages that a call touches are numbered without knowing the lengths: the
// slots of sequence s start at cu_rows[s] / page + 2 s, which leaves room for
// the rows' pages wherever they start. A slot that holds no page ends at once.
#include "cache.cuh"

namespace bdlm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ long long slot_base(const int* cu, int s, int shift) {
    return ((long long)__ldg(cu + s) >> shift) + 2LL * s;
}

// Block-wide check of every sequence; one thread writes the header.
__device__ void check_rows(const CacheWriteArgs& a) {
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0x7fffffff;
    __syncthreads();
    for (int s = threadIdx.x; s < a.c.n_seqs; s += kThreads) {
        const SeqRows r = seq_rows(a.c, a.cu_rows, nullptr, a.total_rows, s);
        bool bad = !r.ok;
        if (r.ok && r.rows > 0)
            for (int p = r.pos0 >> a.c.page_shift; p <= (r.len - 1) >> a.c.page_shift; ++p) {
                const int id = __ldg(a.c.table + (long long)s * a.c.max_pages + p);
                bad = bad || id < 0 || id >= a.c.n_pages;
            }
        if (bad) atomicMin(&s_bad, s);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.hdr->error = s_bad == 0x7fffffff ? DEV_OK : DEV_CHECK;
        a.hdr->info = s_bad == 0x7fffffff ? 0 : s_bad;
    }
}

// eight e4m3 codes of x * inv; values that are not finite become NaN
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        if (!is_finite(x[2 * i])) w[i] = (w[i] & 0xff00u) | 0x7fu;
        if (!is_finite(x[2 * i + 1])) w[i] = (w[i] & 0x00ffu) | 0x7f00u;
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

__device__ __forceinline__ void decode8(uint2 c, float scale, float (&x)[8]) {
    const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[i], __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * i] = f.x * scale;
        x[2 * i + 1] = f.y * scale;
    }
}

// V: 16-byte loads of new rows per thread (page * d / 2048, at least 1)
template <int V>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheWriteArgs a) {
    const CacheView& c = a.c;
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0 && blockIdx.z == 0) check_rows(a);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31;
    // the sequence of this slot: the last s with slot_base(s) <= slot, 32 ways at a time
    const long long slot = blockIdx.x;
    int lo = 0, hi = c.n_seqs;  // in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int probe = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, probe < hi && slot_base(a.cu_rows, probe, c.page_shift) <= slot);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        hi = imin(hi, lo + step);
    }
    const int s = lo;
    const SeqRows r = seq_rows(c, a.cu_rows, nullptr, a.total_rows, s);
    if (!r.ok || r.rows <= 0) return;
    const long long j = slot - slot_base(a.cu_rows, s, c.page_shift);
    const long long page_no = (r.pos0 >> c.page_shift) + j;
    if (j < 0 || page_no > (r.len - 1) >> c.page_shift) return;
    const int id = __ldg(c.table + (long long)s * c.max_pages + page_no);
    if (id < 0 || id >= c.n_pages) return;

    const int head = blockIdx.y, D = c.D;
    const __nv_bfloat16* src = blockIdx.z ? a.v_new : a.k_new;
    const long long unit = (long long)id * c.Hk + head;
    uint8_t* dst = (blockIdx.z ? c.v : c.k) + unit * c.page * D;
    float* scale_at = (blockIdx.z ? c.v_scale : c.k_scale) + unit;
    const int first = (int)(page_no << c.page_shift);  // position of the page's row 0
    const int per_row = D / 8;
    const float was = *scale_at;

    float x[V][8];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int chunk = tid + i * kThreads, row = chunk / per_row, col = chunk % per_row * 8;
        const int pos = first + row;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
        if (row < c.page && pos < r.len) {
            if (pos >= r.pos0) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(
                    src + ((long long)(r.row0 + pos - r.pos0) * c.Hk + head) * D + col));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[i][2 * e] = __uint_as_float(w[e] << 16);
                    x[i][2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                }
            } else {
                decode8(*reinterpret_cast<const uint2*>(dst + row * D + col), was, x[i]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, is_finite(x[i][e]) ? fabsf(x[i][e]) : 0.f);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    __shared__ float s_max[kThreads / 32];
    if (lane == 0) s_max[tid >> 5] = amax;
    __syncthreads();  // also: every thread has read the old scale and the kept rows
    amax = s_max[lane & (kThreads / 32 - 1)];
#pragma unroll
    for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = pow2_scale(amax);
    const float inv = 1.f / scale;  // exact: 2^-126 <= scale <= 2^120
    if (tid == 0) *scale_at = scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int chunk = tid + i * kThreads, row = chunk / per_row, col = chunk % per_row * 8;
        const int pos = first + row;
        if (row < c.page && pos < r.len && (pos >= r.pos0 || scale != was))
            *reinterpret_cast<uint2*>(dst + row * D + col) = encode8(x[i], inv);
    }
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t st, int* launches) {
    const long long slots = ((long long)a.total_rows >> a.c.page_shift) + 2LL * a.c.n_seqs + 1;
    const dim3 grid((unsigned)(slots + 1), (unsigned)a.c.Hk, 2);
    switch (a.c.page * a.c.D / (8 * kThreads)) {
        case 0:
        case 1: cache_write_kernel<1><<<grid, kThreads, 0, st>>>(a); break;
        case 2: cache_write_kernel<2><<<grid, kThreads, 0, st>>>(a); break;
        case 4: cache_write_kernel<4><<<grid, kThreads, 0, st>>>(a); break;
        default: cache_write_kernel<8><<<grid, kThreads, 0, st>>>(a); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace bdlm
