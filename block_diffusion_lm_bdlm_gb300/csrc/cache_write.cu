// cache_write.cu - quantises new key and value rows into the pages of the cache.
//
// A CTA takes one touched page, and of its 2 Hk blocks of page x d values (a kv
// head of K or of V) one or more. A block is held in registers from its one
// read to its one write: rows of the page before the sequence's first new row
// are read back (code * scale), the amax over both gives the new power-of-two
// scale (see pow2_scale), and every value is stored as x / s, rounded once to
// nearest even: the division by a power of two is exact, so the codes are those
// of the definition bit by bit. Kept rows are stored again only where the scale
// has changed.
//
// Bound: memory (2 bytes read and 1 written per value), at small calls the
// latency of offsets, lengths and table in turn. A row of one head is only
// 2 d bytes, so CTAs that run together take the heads of one page, whose rows
// are consecutive bytes (8 prompts of 69500 rows in all, 8 heads, d = 128, page
// 128: 232 us with a page's heads far apart in the grid, 101 side by side, 74
// with all that follows). While a block is
// quantised the next one's rows are on their way, and a page that is new as a
// whole is taken without bounds; its maxima are taken on packed bf16 bits, and
// values that are not finite are looked for only where the maximum says that
// there are some (instruction issue was the limit before). 8 prompts of 8192
// rows take 63 us with 64-row pages (97 before those two), 69 with 128, 71 with
// 16: 6.4, 5.8, 5.6 TB/s of the 403 MB that must move (a copy of them: 59 us).
// 16 blocks of 32 rows take 4.1 us.
//
// The pages that a call touches are numbered without knowing the lengths: the
// slots of sequence s start at cu_rows[s] / page + 2 s, which leaves room for
// the rows' pages wherever they start. A slot that holds no page ends at once.
#include "cache.cuh"

namespace bdlm {
namespace {

constexpr int kV = 4;
// A CTA takes more blocks of its page while as many threads as this per SM remain: half and twice as many take 66.3 and
// 63.9 instead of 64.9 us for 8 prompts of 8192 rows, but 10.3 and 11.0 instead of 9.7 us for 64 blocks of 32 rows that
// begin inside a page, and 12.6 and 12.7 instead of 11.4 us for 256 blocks of 32 rows.
constexpr int kThreadsPerSm = 2048;
constexpr uint32_t kInf = 0x7f800000u;

__device__ __forceinline__ long long slot_base(const int* cu, int s, int shift) {
    return ((long long)__ldg(cu + s) >> shift) + 2LL * s;
}

// Block-wide check of every sequence, a thread for each, and a warp for each that has many pages; one thread writes the
// header.
template <int T>
__device__ void check_rows(const CacheWriteArgs& a) {
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0x7fffffff;
    __syncthreads();
    constexpr int kFew = 4;
    const int lane = threadIdx.x & 31;
    for (int s0 = 0; s0 < a.c.n_seqs; s0 += T) {
        const int s = s0 + threadIdx.x;
        int first = 0, n = 0;  // the touched pages
        if (s < a.c.n_seqs) {
            const SeqRows r = seq_rows(a.c, a.cu_rows, nullptr, a.total_rows, s);
            if (!r.ok) atomicMin(&s_bad, s);
            first = r.pos0 >> a.c.page_shift;
            if (r.ok && r.rows > 0) n = ((r.len - 1) >> a.c.page_shift) - first + 1;
        }
        const int* ids = a.c.table + (long long)s * a.c.max_pages + first;
        bool bad = false;
        if (n <= kFew)
            for (int p = 0; p < n; ++p) bad = bad || (unsigned)__ldg(ids + p) >= (unsigned)a.c.n_pages;
        if (bad) atomicMin(&s_bad, s);
        for (unsigned todo = __ballot_sync(0xffffffffu, n > kFew); todo; todo &= todo - 1) {
            const int src = __ffs(todo) - 1, m = __shfl_sync(0xffffffffu, n, src);
            const int* row = reinterpret_cast<const int*>(__shfl_sync(0xffffffffu, reinterpret_cast<long long>(ids), src));
            bad = false;
#pragma unroll 8
            for (int p = lane; p < m; p += 32) bad = bad || (unsigned)__ldg(row + p) >= (unsigned)a.c.n_pages;
            if (bad) atomicMin(&s_bad, s0 + (int)(threadIdx.x & ~31u) + src);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.hdr->error = s_bad == 0x7fffffff ? DEV_OK : DEV_CHECK;
        a.hdr->info = s_bad == 0x7fffffff ? 0 : s_bad;
    }
}

// Eight e4m3 codes of x * inv. Values that are not finite become NaN, where
// `some` says that there may be any.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv, bool some) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    if (some)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!is_finite(x[2 * i])) w[i] = (w[i] & 0xff00u) | 0x7fu;
            if (!is_finite(x[2 * i + 1])) w[i] = (w[i] & 0x00ffu) | 0x7f00u;
        }
    return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

// A chunk of eight values as it was loaded: bf16 (a new row), or e4m3 codes in
// x and y with the page's old scale (a kept one).
__device__ __forceinline__ void values8(uint4 u, bool kept, float scale, float (&x)[8]) {
    if (kept) {
        const uint32_t w[4] = {u.x & 0xffffu, u.x >> 16, u.y & 0xffffu, u.y >> 16};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[i], __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            x[2 * i] = f.x * scale;
            x[2 * i + 1] = f.y * scale;
        }
    } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ uint32_t umax(uint32_t x, uint32_t y) { return x > y ? x : y; }

// The CTA's largest x; one barrier.
template <int T>
__device__ __forceinline__ uint32_t cta_max(uint32_t x, uint32_t* buf) {
    x = __reduce_max_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, buf[threadIdx.x & (T / 32 - 1)]);
}

__device__ __forceinline__ void rotate(uint4 (&u)[kV]) {
    const uint4 w = u[0];
#pragma unroll
    for (int e = 0; e + 1 < kV; ++e) u[e] = u[e + 1];
    u[kV - 1] = w;
}

// T threads with kV chunks of eight values each: T = page * d / 32. A CTA takes `per_cta` of the 2 Hk (head, K or V) of a
// page, one after the other. (Registers for 1024, 1280, 1536 threads per SM: 64.9, 62.6, 66.8 us for 8 prompts of 8192
// rows and 64-row pages; 70, 87 us for 1024, 1280 and 16-row ones.)
template <int T>
__global__ void __launch_bounds__(T, (T >= 128 ? 1280 : 1024) / T) cache_write_kernel(const CacheWriteArgs a, int per_cta) {
    const CacheView& c = a.c;
    if (blockIdx.x == 0) {
        check_rows<T>(a);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31;
    const unsigned parts = 2u * c.Hk / (unsigned)per_cta;
    const long long slot = (blockIdx.x - 1) / parts;
    const int kind0 = (int)(blockIdx.x - 1 - (unsigned)slot * parts) * per_cta;
    // the sequence of this slot: the last s with slot_base(s) <= slot, 32 ways at a time
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

    const int D = c.D, row_shift = D == 128 ? 4 : 3;   // 2^row_shift chunks are a row
    const int first = (int)(page_no << c.page_shift);  // position of the page's row 0
    const int kept = imax(0, r.pos0 - first);          // rows of the page that stay
    const int rows = imin(c.page, r.len - first);      // and that are there in the end
    const bool whole = kept == 0 && rows == c.page;    // no row is missing (the same for the whole CTA)
    // chunk i of the thread is at row row0 + i * step, columns col .. col + 7: 8 T i bytes behind its first one in the page
    const int row0 = tid >> row_shift, col = (tid & ((1 << row_shift) - 1)) * 8, step = T >> row_shift;
    const int src_step = step * c.Hk * D;
    const long long src0 = (long long)(r.row0 + first - r.pos0 + row0) * c.Hk * D + col;
    const __nv_bfloat16 *k_src = a.k_new + src0, *v_src = a.v_new + src0;

    auto fetch = [&](int kind, uint4 (&u)[kV]) {
        const __nv_bfloat16* src = (kind & 1 ? v_src : k_src) + (kind >> 1) * D;
        if (whole) {
#pragma unroll
            for (int i = 0; i < kV; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(src + (long long)i * src_step));
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int row = row0 + i * step;
                u[i] = make_uint4(0, 0, 0, 0);
                if (row >= kept && row < rows) u[i] = __ldg(reinterpret_cast<const uint4*>(src + (long long)i * src_step));
            }
        }
    };
    uint4 next[kV];
    fetch(kind0, next);
    if (id < 0 || id >= c.n_pages) return;
    __shared__ uint32_t s_max[2][T / 32];
    const long long unit0 = (long long)id * c.Hk;
    uint8_t *k_dst = c.k + unit0 * c.page * D + tid * 8, *v_dst = c.v + unit0 * c.page * D + tid * 8;
    // one (head, K or V) from u
    auto item = [&](int kind, uint32_t* s_buf, uint4 (&u)[kV]) {
        uint8_t* dst = (kind & 1 ? v_dst : k_dst) + (kind >> 1) * c.page * D;
        float* scale_at = (kind & 1 ? c.v_scale : c.k_scale) + unit0 + (kind >> 1);
        float was = 1.f;
        uint32_t top = 0;  // the largest |x| as bits, which order as the values do; above kInf: NaN
        if (kept == 0) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const uint32_t m = __vmaxu2(__vmaxu2(u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu),
                                            __vmaxu2(u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu));
                top = __vmaxu2(top, m);
            }
            top = umax(top << 16, top & 0xffff0000u);
        } else {
            was = *scale_at;
#pragma unroll 1
            for (int i = 0; i < kV; ++i) {
                const int row = row0 + i * step;
                if (row < kept) {
                    const uint2 w = *reinterpret_cast<const uint2*>(dst + i * 8 * T);
                    u[0] = make_uint4(w.x, w.y, 0, 0);
                }
                float x[8];
                values8(u[0], row < kept, was, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = umax(top, __float_as_uint(x[e]) & 0x7fffffffu);
                rotate(u);
            }
        }
        top = cta_max<T>(top, s_buf);  // also: every thread has read the old scale and the kept rows
        const bool some = top >= kInf;
        if (some) {  // the largest of the finite ones
            top = 0;
#pragma unroll 1
            for (int i = 0; i < kV; ++i) {
                float x[8];
                values8(u[0], row0 + i * step < kept, was, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = umax(top, is_finite(x[e]) ? __float_as_uint(x[e]) & 0x7fffffffu : 0u);
                rotate(u);
            }
            __syncthreads();  // s_buf has been read
            top = cta_max<T>(top, s_buf);
        }
        const float scale = pow2_scale(__uint_as_float(top));
        const float inv = __uint_as_float(0x7f000000u - __float_as_uint(scale));  // 1 / scale: 2^-126 <= scale <= 2^120
        if (tid == 0) *scale_at = scale;
        if (whole && !some) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                float x[8];
                values8(u[i], false, 1.f, x);
                *reinterpret_cast<uint2*>(dst + i * 8 * T) = encode8(x, inv, false);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kV; ++i) {
                const int row = row0 + i * step;
                if (row < rows && (row >= kept || scale != was)) {
                    float x[8];
                    values8(u[0], row < kept, was, x);
                    *reinterpret_cast<uint2*>(dst + i * 8 * T) = encode8(x, inv, true);
                }
                rotate(u);
            }
        }
    };
    // two at a time, so that the rows of the next one come in without moving
#pragma unroll 1
    for (int k = 0; k < per_cta; k += 2) {
        uint4 u[kV];
        if (k + 1 < per_cta) fetch(kind0 + k + 1, u);
        item(kind0 + k, s_max[0], next);
        if (k + 1 == per_cta) break;
        if (k + 2 < per_cta) fetch(kind0 + k + 2, next);
        item(kind0 + k + 1, s_max[1], u);
    }
}

template <int T>
void launch(const CacheWriteArgs& a, long long slots, int per_cta, cudaStream_t st) {
    cache_write_kernel<T><<<(unsigned)(slots * (2 * a.c.Hk / per_cta) + 1), T, 0, st>>>(a, per_cta);
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs& a, int num_sms, cudaStream_t st, int* launches) {
    const long long slots = ((long long)a.total_rows >> a.c.page_shift) + 2LL * a.c.n_seqs + 1;
    const int threads = a.c.page * a.c.D / (8 * kV);
    int per_cta = 1;
    while (2 * a.c.Hk % (2 * per_cta) == 0 &&
           slots * (2 * a.c.Hk / (2 * per_cta)) * threads >= (long long)kThreadsPerSm * num_sms)
        per_cta *= 2;
    if (slots * (2 * a.c.Hk / per_cta) >= 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    switch (threads) {
        case 32: launch<32>(a, slots, per_cta, st); break;
        case 64: launch<64>(a, slots, per_cta, st); break;
        case 128: launch<128>(a, slots, per_cta, st); break;
        case 256: launch<256>(a, slots, per_cta, st); break;
        default: launch<512>(a, slots, per_cta, st); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace bdlm
