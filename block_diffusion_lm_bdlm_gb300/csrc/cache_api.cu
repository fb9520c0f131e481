// cache_api.cu - the C ABI of the paged 8-bit cache (include/bdlm.h): host-side
// validation, workspace carving and launches, as in bdlm_api.cu.
#include <cmath>
#include <cstdint>

#include "bdlm.h"
#include "cache.cuh"

using namespace bdlm;

namespace {

constexpr long long kMaxRows = 1LL << 30;   // row indices and positions stay in int32
constexpr int kMaxSeqs = 1 << 16;
constexpr int kMaxPages = 1 << 26;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool good_ptr(const void* p, uintptr_t a) { return p && aligned(p, a); }
bool overlap(const void* x, size_t nx, const void* y, size_t ny) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return x && y && a < b + ny && b < a + nx;
}
bool supported_d(int d) { return d == 64 || d == 128; }

// Checks the cache and fills the kernels' view of its layer `layer`.
int view_of(const bdlm_cache* c, int layer, CacheView* w) {
    if (!c || c->reserved != 0) return BDLM_ERR_INVALID_ARG;
    if (!good_ptr(c->k, 16) || !good_ptr(c->v, 16) || !good_ptr(c->k_scale, 4) || !good_ptr(c->v_scale, 4) ||
        !good_ptr(c->table, 4) || !good_ptr(c->lens, 4))
        return BDLM_ERR_INVALID_ARG;
    if (c->n_layers < 1 || layer < 0 || layer >= c->n_layers || c->n_pages < 1 || c->n_pages > kMaxPages ||
        c->kv_heads < 1 || c->kv_heads > 256 || c->n_seqs < 1 || c->n_seqs > kMaxSeqs || c->max_pages < 1)
        return BDLM_ERR_INVALID_ARG;
    if (!supported_d(c->head_dim)) return BDLM_ERR_UNSUPPORTED;
    int shift = 0;
    switch (c->page) {
        case 16: shift = 4; break;
        case 32: shift = 5; break;
        case 64: shift = 6; break;
        case 128: shift = 7; break;
        default: return BDLM_ERR_UNSUPPORTED;
    }
    if (((long long)c->max_pages << shift) > kMaxRows) return BDLM_ERR_INVALID_ARG;
    if ((long long)c->n_pages * c->kv_heads > (1LL << 30)) return BDLM_ERR_INVALID_ARG;
    const size_t heads = (size_t)c->n_pages * c->kv_heads;
    const size_t codes = heads * c->page * c->head_dim;
    w->k = static_cast<uint8_t*>(c->k) + layer * codes;
    w->v = static_cast<uint8_t*>(c->v) + layer * codes;
    w->k_scale = c->k_scale + layer * heads;
    w->v_scale = c->v_scale + layer * heads;
    w->table = c->table;
    w->lens = c->lens;
    w->n_layers = c->n_layers;
    w->n_pages = c->n_pages;
    w->page = c->page;
    w->Hk = c->kv_heads;
    w->D = c->head_dim;
    w->n_seqs = c->n_seqs;
    w->max_pages = c->max_pages;
    w->page_shift = shift;
    return BDLM_OK;
}

// Does an int32 array of a page call lie in the table or the lengths, which the call writes while it reads the array?
bool in_table(const CacheView& c, const void* p, size_t n) {
    return overlap(p, 4 * n, c.table, 4 * (size_t)c.n_seqs * c.max_pages);
}
bool in_lens(const CacheView& c, const void* p, size_t n) { return overlap(p, 4 * n, c.lens, 4 * (size_t)c.n_seqs); }

int check_workspace(const void* ws, size_t have, size_t need) {
    return ws && aligned(ws, 256) && need > 0 && have >= need ? BDLM_OK : BDLM_ERR_WORKSPACE;
}

int run_pages(const CachePagesArgs& args, void* workspace, size_t workspace_bytes, bdlm_stream_t stream) {
    CachePagesArgs a = args;
    const int st = check_workspace(workspace, workspace_bytes, bdlm_cache_pages_workspace_bytes(a.c.n_pages, a.c.n_seqs));
    if (st != BDLM_OK) return st;
    a.hdr = static_cast<WsHeader*>(workspace);
    a.scratch = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + sizeof(WsHeader));
    const int sms = device_sms();
    int launches = 0;
    if (sms <= 0 || launch_cache_pages(a, sms, reinterpret_cast<cudaStream_t>(stream), &launches) != cudaSuccess)
        return BDLM_ERR_CUDA;
    set_last_launches(launches);
    return BDLM_OK;
}

// Checks the arguments that the attention calls have in common and fills the kernels'.
int attn_args(const bdlm_cache* cache, int layer, const void* q, void* o, float* lse, int64_t total_rows, int heads, int block,
              const int32_t* cu_rows, const int32_t* q_pos, float softmax_scale, int o_dtype, CacheAttnArgs* a) {
    const int st = view_of(cache, layer, &a->c);
    if (st != BDLM_OK) return st;
    if (!good_ptr(q, 16) || !good_ptr(o, 16) || !good_ptr(lse, 4) || !good_ptr(cu_rows, 4) || !aligned(q_pos, 4))
        return BDLM_ERR_INVALID_ARG;
    if (total_rows <= 0 || total_rows > kMaxRows || heads <= 0 || heads % cache->kv_heads != 0 || block <= 0)
        return BDLM_ERR_INVALID_ARG;
    if ((long long)total_rows * (heads / cache->kv_heads) > kMaxRows) return BDLM_ERR_INVALID_ARG;
    if (o_dtype != BDLM_BF16 && o_dtype != BDLM_F32) return BDLM_ERR_INVALID_ARG;
    a->q = static_cast<const __nv_bfloat16*>(q);
    a->o = o_dtype == BDLM_F32 ? nullptr : static_cast<__nv_bfloat16*>(o);
    a->o_f32 = o_dtype == BDLM_F32 ? static_cast<float*>(o) : nullptr;
    a->lse = lse;
    a->cu_rows = cu_rows;
    a->q_pos = q_pos;
    a->total_rows = (int)total_rows;
    a->H = heads;
    a->G = heads / cache->kv_heads;
    a->block = block;
    a->scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)cache->head_dim)) * 1.4426950408889634f;
    return BDLM_OK;
}

// The workspace holds the header, with runs the two planes, and the shares' records and slots.
int run_attn(CacheAttnArgs& a, void* workspace, size_t workspace_bytes, size_t need, bdlm_stream_t stream) {
    const int st = check_workspace(workspace, workspace_bytes, need);
    if (st != BDLM_OK) return st;
    a.hdr = static_cast<WsHeader*>(workspace);
    a.scratch = static_cast<uint8_t*>(workspace) + sizeof(WsHeader);
    if (a.runs) {
        a.planes = reinterpret_cast<float*>(a.scratch);
        a.call_tiles = 32.f / imin(a.c.n_seqs, a.total_rows);
        a.plane_rows = (int)cache_attn_plane_rows(a.total_rows, a.G, a.c.n_seqs);
        a.scratch += cache_attn_plane_bytes(a.plane_rows, a.c.Hk, a.c.D);
    }
    const int sms = device_sms();
    int launches = 0;
    const auto launch = a.runs ? launch_cache_attn_shared : launch_cache_attn;
    if (sms <= 0 || launch(a, sms, reinterpret_cast<cudaStream_t>(stream), &launches) != cudaSuccess) return BDLM_ERR_CUDA;
    set_last_launches(launches);
    return BDLM_OK;
}

}  // namespace

extern "C" {

size_t bdlm_cache_write_workspace_bytes(void) { return sizeof(WsHeader); }

int bdlm_cache_write(const bdlm_cache* cache, int32_t layer, const void* k_new, const void* v_new, int64_t total_rows,
                     const int32_t* cu_rows, void* workspace, size_t workspace_bytes, bdlm_stream_t stream) {
    set_last_launches(0);
    CacheWriteArgs a{};
    int st = view_of(cache, layer, &a.c);
    if (st != BDLM_OK) return st;
    if (!good_ptr(k_new, 16) || !good_ptr(v_new, 16) || !good_ptr(cu_rows, 4)) return BDLM_ERR_INVALID_ARG;
    if (total_rows <= 0 || total_rows > kMaxRows) return BDLM_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, bdlm_cache_write_workspace_bytes());
    if (st != BDLM_OK) return st;
    a.k_new = static_cast<const __nv_bfloat16*>(k_new);
    a.v_new = static_cast<const __nv_bfloat16*>(v_new);
    a.cu_rows = cu_rows;
    a.total_rows = (int)total_rows;
    a.hdr = static_cast<WsHeader*>(workspace);
    const int sms = device_sms();
    int launches = 0;
    if (sms <= 0 || launch_cache_write(a, sms, reinterpret_cast<cudaStream_t>(stream), &launches) != cudaSuccess)
        return BDLM_ERR_CUDA;
    set_last_launches(launches);
    return BDLM_OK;
}

size_t bdlm_cache_attn_fwd_workspace_bytes(int64_t total_rows, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                           int32_t n_seqs) {
    if (total_rows <= 0 || total_rows > kMaxRows || heads <= 0 || kv_heads <= 0 || kv_heads > 256 ||
        heads % kv_heads != 0 || !supported_d(head_dim) || n_seqs < 1 || n_seqs > kMaxSeqs)
        return 0;
    return sizeof(WsHeader) + cache_attn_scratch_bytes(total_rows, heads, kv_heads, head_dim, n_seqs);
}

int bdlm_cache_attn_fwd(const bdlm_cache* cache, int32_t layer, const void* q, void* o, float* lse, int64_t total_rows,
                        int32_t heads, int32_t block, const int32_t* cu_rows, const int32_t* q_pos,
                        float softmax_scale, int32_t o_dtype, void* workspace, size_t workspace_bytes,
                        bdlm_stream_t stream) {
    set_last_launches(0);
    CacheAttnArgs a{};
    const int st = attn_args(cache, layer, q, o, lse, total_rows, heads, block, cu_rows, q_pos, softmax_scale, o_dtype, &a);
    if (st != BDLM_OK) return st;
    return run_attn(a, workspace, workspace_bytes,
                    bdlm_cache_attn_fwd_workspace_bytes(total_rows, heads, cache->kv_heads, cache->head_dim, cache->n_seqs), stream);
}

size_t bdlm_cache_attn_shared_fwd_workspace_bytes(int64_t total_rows, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                                  int32_t n_seqs) {
    const size_t alone = bdlm_cache_attn_fwd_workspace_bytes(total_rows, heads, kv_heads, head_dim, n_seqs);
    if (!alone) return 0;
    return cache_attn_plane_bytes(cache_attn_plane_rows(total_rows, heads / kv_heads, n_seqs), kv_heads, head_dim) + alone;
}

int bdlm_cache_attn_shared_fwd(const bdlm_cache* cache, int32_t layer, const void* q, void* o, float* lse,
                               int64_t total_rows, int32_t heads, int32_t block, const int32_t* cu_rows,
                               const int32_t* q_pos, const int32_t* runs, float softmax_scale, int32_t o_dtype,
                               void* workspace, size_t workspace_bytes, bdlm_stream_t stream) {
    set_last_launches(0);
    CacheAttnArgs a{};
    const int st = attn_args(cache, layer, q, o, lse, total_rows, heads, block, cu_rows, q_pos, softmax_scale, o_dtype, &a);
    if (st != BDLM_OK) return st;
    if (!good_ptr(runs, 4)) return BDLM_ERR_INVALID_ARG;
    a.runs = runs;
    return run_attn(a, workspace, workspace_bytes,
                    bdlm_cache_attn_shared_fwd_workspace_bytes(total_rows, heads, cache->kv_heads, cache->head_dim,
                                                               cache->n_seqs), stream);
}

size_t bdlm_cache_prefixes_workspace_bytes(int32_t n_seqs) {
    if (n_seqs < 1 || n_seqs > cache_prefixes_most_seqs()) return 0;
    return sizeof(WsHeader) + cache_prefixes_scratch_bytes(n_seqs);
}

int bdlm_cache_prefixes(const bdlm_cache* cache, int64_t total_rows, const int32_t* cu_rows, const int32_t* q_pos,
                        int32_t* runs, void* workspace, size_t workspace_bytes, bdlm_stream_t stream) {
    set_last_launches(0);
    CachePrefixArgs a{};
    int st = view_of(cache, 0, &a.c);
    if (st != BDLM_OK) return st;
    if (!good_ptr(cu_rows, 4) || !aligned(q_pos, 4) || !good_ptr(runs, 4)) return BDLM_ERR_INVALID_ARG;
    if (total_rows < 0 || total_rows > kMaxRows) return BDLM_ERR_INVALID_ARG;
    const size_t n = a.c.n_seqs;
    if (in_table(a.c, runs, 3 * n) || in_lens(a.c, runs, 3 * n) || overlap(runs, 12 * n, cu_rows, 4 * (n + 1)) ||
        overlap(runs, 12 * n, q_pos, 4 * n))
        return BDLM_ERR_INVALID_ARG;
    if (a.c.n_seqs > cache_prefixes_most_seqs()) return BDLM_ERR_UNSUPPORTED;
    st = check_workspace(workspace, workspace_bytes, bdlm_cache_prefixes_workspace_bytes(a.c.n_seqs));
    if (st != BDLM_OK) return st;
    a.cu_rows = cu_rows;
    a.q_pos = q_pos;
    a.total_rows = (int)total_rows;
    a.runs = runs;
    a.hdr = static_cast<WsHeader*>(workspace);
    a.scratch = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + sizeof(WsHeader));
    int launches = 0;
    if (launch_cache_prefixes(a, reinterpret_cast<cudaStream_t>(stream), &launches) != cudaSuccess) return BDLM_ERR_CUDA;
    set_last_launches(launches);
    return BDLM_OK;
}

size_t bdlm_cache_pages_workspace_bytes(int32_t n_pages, int32_t n_seqs) {
    if (n_pages < 1 || n_pages > kMaxPages || n_seqs < 1 || n_seqs > kMaxSeqs) return 0;
    return sizeof(WsHeader) + cache_pages_scratch_bytes(n_pages, n_seqs);
}

int bdlm_cache_reserve(const bdlm_cache* cache, const int32_t* new_lens, void* workspace, size_t workspace_bytes,
                       bdlm_stream_t stream) {
    set_last_launches(0);
    CachePagesArgs a{};
    const int st = view_of(cache, 0, &a.c);
    if (st != BDLM_OK) return st;
    if (!good_ptr(new_lens, 4)) return BDLM_ERR_INVALID_ARG;
    if (in_table(a.c, new_lens, a.c.n_seqs) || (new_lens != a.c.lens && in_lens(a.c, new_lens, a.c.n_seqs)))
        return BDLM_ERR_INVALID_ARG;
    a.op = PAGES_RESERVE;
    a.new_lens = new_lens;
    return run_pages(a, workspace, workspace_bytes, stream);
}

int bdlm_cache_fork(const bdlm_cache* cache, const int32_t* parents, const int32_t* children, const int32_t* fork_lens,
                    int32_t n, void* workspace, size_t workspace_bytes, bdlm_stream_t stream) {
    set_last_launches(0);
    CachePagesArgs a{};
    const int st = view_of(cache, 0, &a.c);
    if (st != BDLM_OK) return st;
    if (!good_ptr(parents, 4) || !good_ptr(children, 4) || !aligned(fork_lens, 4)) return BDLM_ERR_INVALID_ARG;
    if (n < 1 || n > cache->n_seqs) return BDLM_ERR_INVALID_ARG;
    if (in_table(a.c, parents, n) || in_lens(a.c, parents, n) || in_table(a.c, children, n) || in_lens(a.c, children, n) ||
        in_table(a.c, fork_lens, n))
        return BDLM_ERR_INVALID_ARG;
    a.op = PAGES_FORK;
    a.parents = parents;
    a.children = children;
    a.fork_lens = fork_lens;
    a.n = n;
    return run_pages(a, workspace, workspace_bytes, stream);
}

int bdlm_cache_compact(const bdlm_cache* cache, int32_t* n_live, void* workspace, size_t workspace_bytes,
                       bdlm_stream_t stream) {
    set_last_launches(0);
    CachePagesArgs a{};
    const int st = view_of(cache, 0, &a.c);
    if (st != BDLM_OK) return st;
    if (!aligned(n_live, 4) || in_table(a.c, n_live, 1) || in_lens(a.c, n_live, 1)) return BDLM_ERR_INVALID_ARG;
    a.op = PAGES_COMPACT;
    a.n_live = n_live;
    return run_pages(a, workspace, workspace_bytes, stream);
}

}  // extern "C"
