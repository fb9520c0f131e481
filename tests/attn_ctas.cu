// The attention over the paged cache with a given number of CTAs (the library takes one per SM), for tests that cut the
// same work in other places. Linked with the library's own objects.
#include <cmath>

#include "bdlm.h"
#include "cache.cuh"

extern "C" __attribute__((visibility("default"))) int attn_with_ctas(const bdlm_cache* c, const void* q, void* o,
                                                                     float* lse, long long rows, int heads, int block,
                                                                     const int* cu_rows, int f32, void* ws, int ctas,
                                                                     void* stream) {
    bdlm::CacheAttnArgs a{};
    int shift = 0;
    while ((1 << shift) < c->page) ++shift;
    a.c = {(uint8_t*)c->k, (uint8_t*)c->v, c->k_scale,    c->v_scale,  c->table, c->lens,      c->n_layers,
           c->n_pages,     c->page,        c->kv_heads,   c->head_dim, c->n_seqs, c->max_pages, shift};
    a.q = (const __nv_bfloat16*)q;
    a.o = f32 ? nullptr : (__nv_bfloat16*)o;
    a.o_f32 = f32 ? (float*)o : nullptr;
    a.lse = lse;
    a.cu_rows = cu_rows;
    a.total_rows = (int)rows;
    a.H = heads;
    a.G = heads / c->kv_heads;
    a.block = block;
    a.scale_log2 = 1.4426950408889634f / std::sqrt((float)c->head_dim);
    a.hdr = (bdlm::WsHeader*)ws;
    a.scratch = (uint8_t*)ws + sizeof(bdlm::WsHeader);
    int launches = 0;
    return (int)bdlm::launch_cache_attn(a, ctas, (cudaStream_t)stream, &launches);
}
