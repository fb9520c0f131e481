// cache.cuh - what the kernels of the paged 8-bit cache share: the cache as the
// kernels see it, the e4m3 conversions and the checks of rows and lengths.
//
// A cached value is scale * code, with an e4m3 code (1 sign, 4 exponent, 3
// mantissa bits, largest 448, no infinities, NaN = 0x7f) and one fp32 scale per
// page and kv head.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace bdlm {

constexpr int DEV_NO_PAGES = 7;  // device error word, the value of BDLM_ERR_NO_PAGES

struct CacheView {
    uint8_t* k;  // the layer's pages [n_pages, Hk, page, d] (page calls: layer 0)
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    int* table;
    int* lens;
    int n_layers, n_pages, page, Hk, D, n_seqs, max_pages;
    int page_shift;  // log2(page)
};

// The rows of one sequence in a call.
struct SeqRows {
    int row0, rows;  // rows [row0, row0 + rows) of q / k_new / v_new
    int len;         // positions that the cache holds
    int pos0;        // position of the first row
    bool ok;         // offsets and length are well-formed
};

// Reads and checks sequence s. With q_pos == nullptr the rows are the last
// ones that the sequence holds.
__device__ __forceinline__ SeqRows seq_rows(const CacheView& c, const int* cu_rows, const int* q_pos, int total_rows,
                                            int s) {
    SeqRows r;
    const int a = __ldg(cu_rows + s), b = __ldg(cu_rows + s + 1);
    r.row0 = a;
    r.rows = b - a;
    r.len = __ldg(c.lens + s);
    r.ok = a >= 0 && b >= a && b <= total_rows && (s > 0 || a == 0) && r.len >= 0 &&
           (long long)r.len <= (long long)c.max_pages << c.page_shift;
    if (q_pos) {
        r.pos0 = __ldg(q_pos + s);
        r.ok = r.ok && r.pos0 >= 0 && (long long)r.pos0 + r.rows <= (1LL << 30);
    } else {
        r.pos0 = r.len - r.rows;
        r.ok = r.ok && r.pos0 >= 0;
    }
    return r;
}

// Keys that the row at position p sees: [0, key_end).
__device__ __forceinline__ int key_end(int len, int block, int p) {
    const long long e = ((long long)(p / block) + 1) * block;
    return e < len ? (int)e : len;
}

// The smallest power of two s >= 2^-126 with amax <= 448 s (1 for amax = 0).
// 448 = 1.75 * 2^8, so with amax = m 2^e, 1 <= m < 2, it is 2^(e-8) for
// m <= 1.75 and 2^(e-7) above.
__device__ __forceinline__ float pow2_scale(float amax) {
    if (amax == 0.f) return 1.f;
    const uint32_t b = __float_as_uint(amax);
    int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased exponent of the scale
    return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

__device__ __forceinline__ bool is_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// Internal launch interface.
struct CacheWriteArgs {
    CacheView c;
    const __nv_bfloat16* k_new;
    const __nv_bfloat16* v_new;
    const int* cu_rows;
    int total_rows;
    WsHeader* hdr;
};
struct CacheAttnArgs {
    CacheView c;
    const __nv_bfloat16* q;
    __nv_bfloat16* o;  // bf16 output (o_f32 == nullptr)
    float* o_f32;
    float* lse;
    const int* cu_rows;
    const int* q_pos;
    int total_rows, H, G, block;
    float scale_log2;  // softmax scale * log2(e)
    WsHeader* hdr;
    uint8_t* scratch;  // behind the header
};
enum PageOp : int { PAGES_RESERVE = 0, PAGES_FORK = 1, PAGES_COMPACT = 2 };
struct CachePagesArgs {
    CacheView c;
    int op;
    const int* new_lens;
    const int* parents;
    const int* children;
    const int* fork_lens;
    int n;        // forks
    int* n_live;  // compact: receives the count of live pages
    WsHeader* hdr;
    int* scratch;
};

size_t cache_attn_scratch_bytes(long long total_rows, int H, int Hk, int D, int n_seqs);
size_t cache_pages_scratch_bytes(int n_pages, int n_seqs);
cudaError_t launch_cache_write(const CacheWriteArgs& a, int num_sms, cudaStream_t st, int* launches);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, int num_sms, cudaStream_t st, int* launches);
cudaError_t launch_cache_pages(const CachePagesArgs& a, int num_sms, cudaStream_t st, int* launches);

int device_sms();
void set_last_launches(int n);

}  // namespace bdlm
